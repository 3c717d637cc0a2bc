"""Argument checks of the projections, rotations, the rotary append and the tree attention at the
C ABI, all answered before any HIP call (no GPU needed)."""
import ctypes
import math

import scoring_exact_top_amd as st

GOOD, OFF8, OFF2, WS = (ctypes.c_void_p(x) for x in (1 << 20, (1 << 20) + 8, (1 << 20) + 2, 1 << 30))
L = st.raw_library()


def _matmul(**k):
    g = k.get
    return L.idx_topk_matmul_e4m3(g("x", GOOD), g("xr", 256), g("xs", GOOD), g("group", 128), g("w", GOOD), g("ws", GOOD), g("M", 4), g("N", 64),
                                  g("K", 256), g("type", 0), g("out", GOOD), g("orow", 64), None)


def test_matmul_arguments():
    for bad in ({"x": None}, {"x": OFF8}, {"xs": None}, {"xs": OFF2}, {"w": None}, {"w": OFF8}, {"ws": None}, {"ws": OFF2}, {"out": None},
                {"out": OFF8}, {"M": -1}, {"N": 0}, {"K": 0}, {"K": 8}, {"K": 250}, {"type": 2}, {"type": -1}, {"xr": 8}, {"xr": -16},
                {"orow": 63}, {"orow": -1}):
        assert _matmul(**bad) == -1, bad
    for bad in ({"group": 64}, {"K": (1 << 24) + 16}, {"xr": (1 << 24) + 16}, {"M": 1 << 20, "N": 1 << 20, "orow": 1 << 20}):
        assert _matmul(**bad) == -2, bad
    assert _matmul(M=0) == 0


def _rotate(**k):
    g = k.get
    return L.idx_topk_norm_rotate(g("x", GOOD), g("xt", 1280), g("xh", 128), g("norm", 1), g("w", GOOD), g("b", GOOD), g("eps", 1e-6),
                                  g("pos", GOOD), g("table", GOOD), g("rows", 100), g("at", 64), 0, g("T", 4), g("H", 10), g("D", 128),
                                  g("dtype", 0), g("out", WS), g("ot", 1280), g("oh", 128), g("codes", None), g("scales", None), None)


def test_rotate_arguments():
    for bad in ({"x": None}, {"x": OFF8}, {"w": OFF8}, {"b": OFF8}, {"pos": None}, {"pos": OFF2}, {"table": None}, {"table": OFF8},
                {"out": None}, {"out": OFF8}, {"rows": -1}, {"at": -8}, {"at": 4}, {"at": 72}, {"T": -1}, {"H": 0}, {"D": 56}, {"D": 132},
                {"D": 1032}, {"dtype": 2}, {"norm": 3}, {"norm": -1}, {"eps": -1.0}, {"eps": math.nan}, {"eps": math.inf}, {"xt": 4},
                {"xh": -8}, {"ot": 4}, {"oh": 64}, {"ot": 64}, {"codes": WS, "scales": WS}, {"out": None, "codes": WS},
                {"out": None, "scales": WS}, {"out": None, "codes": OFF8, "scales": WS}, {"out": None, "codes": WS, "scales": OFF2},
                {"norm": 0}, {"norm": 0, "w": None}, {"norm": 0, "b": None},          # a weight or bias without a norm
                {"out": GOOD, "xt": 2560}, {"out": GOOD, "xh": 256}):                 # in place with other strides
        assert _rotate(**bad) == -1, bad
    assert _rotate(T=1 << 30, H=128) == -2
    assert _rotate(T=0) == 0 and _rotate(rows=0) == 0
    assert _rotate(norm=0, w=None, b=None, eps=math.nan, T=0) == 0                    # eps is not looked at


def _append(**k):
    g = k.get
    return L.idx_topk_cache_append_rotary(g("lat", GOOD), g("ls", 576), g("ln", 1), g("lw", GOOD), g("le", 1e-6), 1, g("key", GOOD), g("ks", 128),
                                          g("kn", 2), g("kw", GOOD), g("kb", GOOD), g("ke", 1e-6), g("at", 0), 0, g("slots", GOOD),
                                          g("pos", GOOD), g("table", GOOD), g("rows", 100), g("T", 4), g("dtype", 0), g("lc", GOOD),
                                          g("kc", GOOD), g("sc", GOOD), g("n", 100), g("lo", WS), None)


def test_append_rotary_arguments():
    for bad in ({"lat": None}, {"lc": None}, {"key": None}, {"kc": None}, {"sc": None}, {"lat": OFF8}, {"lc": OFF8}, {"key": OFF8},
                {"kc": OFF8}, {"sc": OFF2}, {"slots": None}, {"slots": OFF2}, {"pos": None}, {"pos": OFF2}, {"table": None}, {"table": OFF8},
                {"lo": OFF8}, {"lw": OFF8}, {"kw": OFF8}, {"kb": OFF8}, {"T": -1}, {"n": -1}, {"rows": -1}, {"ls": 3}, {"ks": -8},
                {"dtype": 9}, {"ln": 2}, {"ln": 3}, {"kn": -1}, {"ln": 0}, {"kn": 0}, {"kn": 0, "kw": None}, {"le": -1.0}, {"ke": math.nan},
                {"at": 4}, {"at": 72}, {"at": -8}, {"lo": GOOD, "ls": 1152}, {"lat": None, "lc": None}):
        assert _append(**bad) == -1, bad
    assert _append(T=0) == 0 and _append(n=0) == 0 and _append(rows=0) == 0


def _tree(**k):
    g = k.get
    return L.idx_topk_latent_tree(g("q", GOOD), g("qs", 576 * 640), g("qt", 576 * 64), g("qh", 576), g("cache", GOOD), g("P", 100),
                                  g("table", GOOD), g("max_pages", 16), g("prefix", GOOD), g("counts", GOOD), g("masks", GOOD), g("ms", 10),
                                  g("B", 4), g("S", 10), g("H", 64), g("scale", 0.1), g("dtype", 1), g("out", GOOD), g("lse", None),
                                  g("ws", WS), g("wsb", 1 << 40), None)


def test_tree_arguments():
    off4 = ctypes.c_void_p((1 << 20) + 4)
    for bad in ({"q": None}, {"q": OFF8}, {"table": None}, {"table": OFF2}, {"prefix": None}, {"prefix": OFF2}, {"counts": OFF2},
                {"masks": None}, {"masks": off4}, {"ms": -1}, {"S": 0}, {"S": 65}, {"B": -1}, {"H": 0}, {"P": -1}, {"max_pages": -1},
                {"scale": 0.0}, {"scale": math.nan}, {"dtype": 2}, {"qt": 12}, {"qs": -8}, {"cache": None}, {"cache": OFF8}, {"out": None},
                {"out": OFF8}, {"lse": OFF2}, {"ws": ctypes.c_void_p((1 << 30) + 64)}):
        assert _tree(**bad) == -1, bad
    assert _tree(H=129) == -2 and _tree(max_pages=1 << 25) == -2 and _tree(B=1 << 20, S=64, H=128) == -2
    assert _tree(ws=None) == -3 and _tree(wsb=16) == -3
    assert _tree(B=0) == 0
    for bad in ((-1, 1, 64, 8), (4, 0, 64, 8), (4, 65, 64, 8), (4, 1, 129, 8), (4, 1, 64, -1)):
        assert st.latent_tree_workspace_bytes(*bad) == 0, bad


def test_tree_workspace_is_bounded():
    """Whatever the batch, nodes, heads and table: the bound that the header states."""
    for B in (0, 1, 2, 16, 100, 256, 300, 1023, 1024, 1025, 5000):
        for S in (1, 7, 16, 17, 33, 50, 64):
            for H in (1, 16, 20, 33, 64, 100, 113, 128):
                for max_pages in (0, 1, 3, 16, 1024, 1 << 20):
                    need = st.latent_tree_workspace_bytes(B, S, H, max_pages)
                    assert 256 <= need <= 132 << 20, (B, S, H, max_pages, need)
