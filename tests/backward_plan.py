"""What archead_backward launches for a shape, from the rules and constants of
csrc/backward.hip (constants are read from the source), so that the tests can
say which kernels their shapes reach."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_quantized_lm_amd", "csrc",
                   "backward.hip")


def _constants():
    text = open(SRC).read()
    c = {n: int(v) for n, v in re.findall(r"\b(k[A-Z]\w+) = (\d+)\b", text)}
    c["kSumRate"] = float(re.search(r"kSumRate = ([\d.e]+)", text).group(1))
    c["kChunkM"] = int(re.search(r"kChunkM = (\d+)", text).group(1))
    kinds = re.search(r"kTiles\[\] = \{(.*?)\};", text).group(1)
    c["kTiles"] = [(int(a), int(b), float(us)) for a, b, us in re.findall(r"\{(\d+), (\d+), ([\d.]+)\}", kinds)]
    return c


C = _constants()


def _up(a, b):
    return -(-a // b)


def _ranges_of(kind, M, tiles, tile_cols, nvc):
    rows, places, us = kind
    t = max(tiles * _up(M, rows), 1)
    at, most = C["kCu"] * places, max(1, nvc // C["kMinChunks"])
    sums = M * tiles * tile_cols * 8 / C["kSumRate"]
    least, best, S = 1e300, 1, 1
    while S <= most and (S == 1 or S * t <= C["kMaxWg"]):
        chunks = _up(nvc, S)
        cost = _up(S * t, at) * (chunks + 2.0) * us + S * sums
        if cost < least * 0.995:
            least, best = cost, S
        if chunks == 1:
            break
        S = _up(nvc, chunks - 1)
    return least, best


def _tiles(V, d, k, r):
    units = _up(k, C["kUnit"]) + _up(r, C["kUnit"])
    return _up(V, C["kVC"]), _up(d, C["kJT"]), units, _up(units * C["kUnit"], C["kLT"])


def _plan(V, d, k, r, M):
    """Rows of a tile, ranges of the low-rank tiles and of dX's."""
    nvc, main, _, low = _tiles(V, d, k, r)
    best, least = None, 1e300
    for kind in C["kTiles"]:
        if (kind[0] == 32) != (M <= 32):
            continue
        a, s_main = _ranges_of(kind, M, main, C["kJT"], nvc)
        b, s_low = _ranges_of(kind, M, low, C["kLT"], nvc) if low else (0.0, 1)
        if a + b < least:
            least, best = a + b, (kind[0], s_low, s_main)
    return best


def launches(V, d, k, r, M, dtype="bfloat16"):
    """Of one part (M up to kChunkM rows): the set of kernel forms launched."""
    _, main, units, low = _tiles(V, d, k, r)
    bm, s_low, s_main = _plan(V, d, k, r, M)
    found = set()
    if low:
        found.add(f"low tiles {bm}, {'full' if low * C['kLT'] == units * C['kUnit'] else 'partly padding'}")

    def groups(S, n_jt):
        return _up(S * _up(M, bm) * n_jt, 8) * 8
    n, everything = groups(s_low, low) if low else 0, (groups(s_low, low) if low else 0) + groups(s_main, main)
    places = C["kCu"] * (2 if bm == 64 else 1)
    if n:
        found.add("one launch" if bm == 32 or everything <= places + places // 2 else "two launches")
    found.add(f"tiles {bm}, {'several ranges' if s_main > 1 else 'one range'}")
    tiles = _up(M, 16) * (d // 16)
    form = "split" if tiles <= 512 else "16 x 16" if M <= 512 else "64 x 64"
    found |= {f"finish {form}", f"tiles {bm}, finish {form}"}
    whole = V >= C["kWide"] * 8 and 10 * M >= 7 * _up(M, C["kCu"]) * C["kCu"]
    found.add(f"convert {'a row' if whole else 'slices'} {dtype}")
    return found


def of_call(V, d, k, r, M, reserved, dtype="bfloat16"):
    """Of a whole call on a head with room for reserved rows."""
    part = min(reserved, C["kChunkM"])
    found = set()
    for m in range(0, M, part):
        found |= launches(V, d, k, r, min(part, M - m), dtype)
    if M > part:
        found.add("parts of kChunkM" if part == C["kChunkM"] else "parts")
    return found


def workspace_bytes(V, d, k, r, reserved):
    """Of a head with room for reserved rows: G in fp16, a few numbers a row, T
    sB in two parts and U, and the ranges' sums of the largest plan."""
    rows = min(reserved, C["kChunkM"])
    nvc, main, _, low = _tiles(V, d, k, r)
    s_low = s_main = 0
    for M in range(1, rows + 1):
        _, a, b = _plan(V, d, k, r, M)
        s_low, s_main = max(s_low, a * M * low * C["kLT"]), max(s_main, b * M * main * C["kJT"])
    core, correction = _up(k, 32) * 32, _up(r, 32) * 32
    parts = [rows * nvc * C["kVC"] * 2, rows * C["kAmaxSlices"] * 4, rows * 4, s_low * 4, rows * core * 2,
             rows * core * 2, rows * correction * 4, s_main * 4]
    return sum(_up(max(p, 16), 256) * 256 for p in parts)
