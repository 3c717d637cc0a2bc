"""Argument checks of the operators around the indexer at the C ABI, all
answered before any HIP call (no GPU needed)."""
import ctypes
import math

import scoring_exact_top_amd as st

GOOD, OFF8, WS, BIG = (ctypes.c_void_p(x) for x in (1 << 20, (1 << 20) + 8, 1 << 30, 0))
L = st.raw_library()


def _selected(**k):
    g = k.get
    return L.idx_topk_latent_selected(g("q", GOOD), g("qt", 576 * 64), g("qh", 576), g("cache", GOOD), g("n", 1000), g("slots", GOOD),
                                      g("K", 2048), g("T", 4), g("H", 64), g("scale", 0.1), g("dtype", 0), g("out", GOOD), None,
                                      g("ws", WS), g("wsb", 1 << 40), None)


def test_selected_arguments():
    for bad in ({"q": None}, {"q": OFF8}, {"cache": OFF8}, {"cache": None}, {"slots": None}, {"out": None}, {"out": OFF8}, {"K": 0},
                {"K": 2049}, {"T": -1}, {"H": 0}, {"n": -1}, {"scale": 0.0}, {"scale": -1.0}, {"scale": math.inf}, {"scale": math.nan},
                {"dtype": 2}, {"qt": 4}, {"qh": -8}, {"ws": ctypes.c_void_p((1 << 30) + 64)}):
        assert _selected(**bad) == -1, bad
    assert _selected(H=129) == -2
    assert _selected(ws=None) == -3
    assert _selected(wsb=16) == -3
    assert _selected(T=0) == 0
    assert st.latent_selected_workspace_bytes(4, 64, 2048) > 0
    for bad in ((-1, 64, 8), (4, 0, 8), (4, 129, 8), (4, 64, 0), (4, 64, 2049)):
        assert st.latent_selected_workspace_bytes(*bad) == 0, bad


def _paged(**k):
    g = k.get
    return L.idx_topk_latent_paged(g("q", GOOD), 576 * 64, g("qt", 576 * 64), g("qh", 576), g("cache", GOOD), g("P", 100), g("table", GOOD),
                                   g("max_pages", 16), g("lens", GOOD), g("B", 4), g("S", 1), g("H", 64), g("scale", 0.1), g("dtype", 1),
                                   g("out", GOOD), None, g("ws", WS), g("wsb", 1 << 40), None)


def test_paged_arguments():
    for bad in ({"q": None}, {"q": OFF8}, {"table": None}, {"lens": None}, {"S": 0}, {"S": 17}, {"B": -1}, {"H": 0}, {"P": -1},
                {"max_pages": -1}, {"scale": 0.0}, {"dtype": -1}, {"qt": 12}, {"ws": ctypes.c_void_p((1 << 30) + 64)}):
        assert _paged(**bad) == -1, bad
    assert _paged(H=129) == -2
    assert _paged(max_pages=1 << 25) == -2
    assert _paged(ws=None) == -3
    assert _paged(B=0) == 0
    assert st.latent_paged_workspace_bytes(16, 1, 128, 1024) > 0
    for bad in ((-1, 1, 64, 8), (4, 0, 64, 8), (4, 17, 64, 8), (4, 1, 129, 8), (4, 1, 64, -1)):
        assert st.latent_paged_workspace_bytes(*bad) == 0, bad


def _expanded(**k):
    g = k.get
    return L.idx_topk_latent_expanded(g("q", GOOD), g("qt", 1920), g("qh", 192), g("kv", GOOD), g("kt", 2560), 256, g("rope", GOOD),
                                      g("rt", 64), g("cq", GOOD), g("ck", GOOD), g("B", 2), g("Tq", 100), g("Tk", 100), g("mq", 60),
                                      g("mk", 60), g("H", 10), g("scale", 0.1), 1, g("dtype", 0), g("out", GOOD), None, g("ws", WS),
                                      g("wsb", 1 << 40), None)


def test_expanded_arguments():
    for bad in ({"q": None}, {"q": OFF8}, {"kv": None}, {"kv": OFF8}, {"rope": None}, {"rope": OFF8}, {"cq": None}, {"ck": None},
                {"out": OFF8}, {"B": -1}, {"Tq": -1}, {"Tk": -1}, {"mq": -1}, {"mk": -1}, {"H": 0}, {"scale": 0.0}, {"dtype": 7}, {"qt": 4},
                {"kt": 2}, {"rt": -64}):
        assert _expanded(**bad) == -1, bad
    assert _expanded(H=129) == -2
    assert _expanded(B=65536) == -2
    assert _expanded(ws=None) == -3
    assert _expanded(B=0) == 0 and _expanded(Tq=0) == 0
    for bad in ((-1, 1, 8, 8, 4), (4, -1, 8, 8, 4), (4, 1, -1, 8, 4), (4, 1, 8, -1, 4), (4, 1, 8, 8, 0), (4, 1, 8, 8, 129)):
        assert st.latent_expanded_workspace_bytes(*bad) == 0, bad


def _norm(**k):
    g = k.get
    return L.idx_topk_norm_quant(g("x", GOOD), g("xs", 256), g("res", GOOD), g("rs", 256), None, g("eps", 1e-6), g("rows", 4), g("width", 256),
                                 g("group", 128), g("dtype", 0), g("codes", GOOD), g("scales", WS), g("ro", None), None)


def test_norm_arguments():
    odd = ctypes.c_void_p((1 << 20) + 1)
    for bad in ({"x": None}, {"x": odd}, {"res": odd}, {"codes": None}, {"scales": None}, {"scales": ctypes.c_void_p((1 << 20) + 2)},
                {"rows": -1}, {"width": 0}, {"width": 16385}, {"width": 200}, {"eps": -1.0}, {"eps": math.inf}, {"eps": math.nan}, {"dtype": 3},
                {"xs": -1}, {"ro": GOOD, "xs": 300}, {"ro": GOOD, "rs": 300}):
        assert _norm(**bad) == -1, bad
    assert _norm(group=64) == -2
    assert _norm(rows=0) == 0


def _append(**k):
    g = k.get
    return L.idx_topk_cache_append(g("lat", GOOD), g("ls", 576), g("key", GOOD), g("ks", 128), g("slots", GOOD), g("T", 4), g("dtype", 0),
                                   g("lc", GOOD), g("kc", GOOD), g("sc", GOOD), g("n", 100), None)


def test_append_arguments():
    for bad in ({"lat": None}, {"lc": None}, {"key": None}, {"kc": None}, {"sc": None}, {"lat": OFF8}, {"lc": OFF8}, {"key": OFF8},
                {"kc": OFF8}, {"slots": None}, {"T": -1}, {"n": -1}, {"ls": 3}, {"ks": -8}, {"dtype": 9}):
        assert _append(**bad) == -1, bad
    assert _append(T=0) == 0 and _append(n=0) == 0
