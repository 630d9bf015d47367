"""Refusals of the serving calls (CPU only: arguments are checked on the host and the
placeholder pointers are never followed)."""
import ctypes

import pytest

from speculative_decoding_tree_04_gb300 import tv

FAKE = 1 << 20


def sample_args(**kw):
    a = tv.SampleArgs()
    a.struct_size = ctypes.sizeof(tv.SampleArgs)
    a.B, a.Q, a.vocab = 2, 9, 1000
    a.logits, a.logits_dt, a.logits_row_stride = FAKE, tv.TV_F32, 1000
    a.parent, a.tokens, a.uniforms = FAKE + (1 << 20), FAKE + (2 << 20), FAKE + (3 << 20)
    a.accept_len, a.path, a.new_tokens = FAKE + (4 << 20), FAKE + (5 << 20), FAKE + (6 << 20)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), tv.TV_ERR_INVALID_ARG),
    (dict(B=-1), tv.TV_ERR_INVALID_ARG),
    (dict(Q=0), tv.TV_ERR_INVALID_ARG),
    (dict(Q=65), tv.TV_ERR_UNSUPPORTED),
    (dict(vocab=0), tv.TV_ERR_INVALID_ARG),
    (dict(vocab=(1 << 18) + 1, logits_row_stride=1 << 19), tv.TV_ERR_UNSUPPORTED),
    (dict(logits_dt=2), tv.TV_ERR_INVALID_ARG),
    (dict(logits_row_stride=999), tv.TV_ERR_INVALID_ARG),
    (dict(logits_row_stride=1 << 60), tv.TV_ERR_INVALID_ARG),
    (dict(logits=None), tv.TV_ERR_INVALID_ARG),
    (dict(logits=FAKE + 2), tv.TV_ERR_INVALID_ARG),
    (dict(uniforms=None), tv.TV_ERR_INVALID_ARG),
    (dict(path=None), tv.TV_ERR_INVALID_ARG),
    (dict(draft_probs=FAKE, draft_row_stride=999, draft_rows=9), tv.TV_ERR_INVALID_ARG),
    (dict(draft_probs=FAKE, draft_row_stride=1000, draft_rows=0), tv.TV_ERR_INVALID_ARG),
    (dict(draft_probs=FAKE, draft_row_stride=1 << 60, draft_rows=9), tv.TV_ERR_INVALID_ARG),
    (dict(draft_probs=FAKE, draft_row_stride=1000, draft_rows=9, draft_mode=2),
     tv.TV_ERR_INVALID_ARG),
    (dict(draft_probs=FAKE, draft_row_stride=1000, draft_rows=8, draft_mode=1),
     tv.TV_ERR_INVALID_ARG),
    (dict(draft_probs=FAKE + 2, draft_row_stride=1000, draft_rows=9), tv.TV_ERR_INVALID_ARG),
    (dict(new_tokens=FAKE + (2 << 20)), tv.TV_ERR_INVALID_ARG),        # in place over tokens
    (dict(path=FAKE + (1 << 20) + 68), tv.TV_ERR_INVALID_ARG),         # parent's last entry
    (dict(accept_len=FAKE + (5 << 20)), tv.TV_ERR_INVALID_ARG),        # and path
    (dict(temperature=FAKE + (4 << 20) + 4), tv.TV_ERR_INVALID_ARG),
    (dict(new_tokens=FAKE + 4 * (17 * 1000 + 999)), tv.TV_ERR_INVALID_ARG),  # the last logit
    (dict(draft_probs=FAKE + (5 << 20) - 4 * 999, draft_row_stride=1000, draft_rows=9),
     tv.TV_ERR_INVALID_ARG),
    (dict(B=0, logits=None), tv.TV_OK),
])
def test_tree_sample_arguments(tvlib, kw, code):
    assert tv.load().tv_tree_sample(ctypes.byref(sample_args(**kw)), None) == code
    assert (code == tv.TV_OK) == (not tv.load().tv_last_error())


def pool(**kw):
    p = tv.PagePool(FAKE, FAKE, FAKE, 8, 16, 100, 64)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), tv.TV_ERR_INVALID_ARG),
    (dict(rows=4097), tv.TV_ERR_UNSUPPORTED),
    (dict(max_pages=0), tv.TV_ERR_INVALID_ARG),
    (dict(num_pages=0), tv.TV_ERR_INVALID_ARG),
    (dict(num_pages=1 << 24), tv.TV_ERR_UNSUPPORTED),
    (dict(page_size=0), tv.TV_ERR_INVALID_ARG),
    (dict(max_pages=1 << 25), tv.TV_ERR_UNSUPPORTED),
    (dict(refcount=None), tv.TV_ERR_INVALID_ARG),
    (dict(page_table=None), tv.TV_ERR_INVALID_ARG),
])
def test_pool_arguments(tvlib, kw, code):
    lib, p = tv.load(), ctypes.byref(pool(**kw))
    assert lib.tv_pages_workspace_size(p) == 0
    assert lib.tv_pages_reserve(p, FAKE, FAKE, FAKE, None, FAKE, 1 << 20, None) == code
    assert lib.tv_pages_fork(p, FAKE, FAKE, None, None) == code
    assert lib.tv_pages_release(p, FAKE, None, None) == code
    assert lib.tv_pages_compact(p, FAKE, FAKE, None, FAKE, 1 << 20, None) == code
    assert lib.tv_last_error()


def test_pool_pointers_and_workspace(tvlib):
    lib, p = tv.load(), ctypes.byref(pool())
    need = lib.tv_pages_workspace_size(p)
    assert need > 0 and need % 256 == 0
    bad, short = tv.TV_ERR_INVALID_ARG, tv.TV_ERR_WORKSPACE
    assert lib.tv_pages_reserve(None, FAKE, FAKE, FAKE, None, FAKE, need, None) == bad
    assert lib.tv_pages_reserve(p, None, FAKE, FAKE, None, FAKE, need, None) == bad
    assert lib.tv_pages_reserve(p, FAKE, FAKE, FAKE, None, None, need, None) == short
    assert lib.tv_pages_reserve(p, FAKE, FAKE, FAKE, None, FAKE + 16, need, None) == short
    assert lib.tv_pages_reserve(p, FAKE, FAKE, FAKE, None, FAKE, need - 1, None) == short
    assert lib.tv_pages_fork(p, None, FAKE, None, None) == bad
    assert lib.tv_pages_release(p, None, None, None) == bad
    assert lib.tv_pages_compact(p, None, FAKE, None, FAKE, need, None) == bad
    assert lib.tv_pages_compact(p, FAKE, FAKE, None, FAKE, need - 1, None) == short


def test_pages_copy_arguments(tvlib):
    ok = dict(c=FAKE, k=FAKE, dt=1, cs=512, ks=64, dl=512, dr=64, layers=2, cl=1 << 20,
              kl=1 << 18, ps=64, rows=6400, lst=FAKE, n=4)

    def call(**kw):
        p = dict(ok, **kw)
        return tv.load().tv_pages_copy(p["c"], p["k"], p["dt"], p["cs"], p["ks"], p["dl"],
                                       p["dr"], p["layers"], p["cl"], p["kl"], p["ps"],
                                       p["rows"], p["lst"], None, p["n"], None, None)

    assert call(n=0) == tv.TV_OK
    for kw in (dict(c=None), dict(k=None), dict(lst=None), dict(dt=3), dict(dl=0), dict(dr=-1),
               dict(cs=511), dict(ks=56), dict(dl=508), dict(dr=4), dict(cs=516), dict(ks=68),
               dict(c=FAKE + 8), dict(k=FAKE + 8), dict(layers=0), dict(cl=-8), dict(cl=1004),
               dict(ps=0), dict(rows=-1), dict(n=-1)):
        assert call(**kw) == tv.TV_ERR_INVALID_ARG, kw
    assert call(ps=65537) == tv.TV_ERR_UNSUPPORTED


def test_new_status_has_a_text(tvlib):
    assert tv.load().tv_status_string(tv.TV_ERR_NO_PAGES) == b"too few free pages"


def prefill_args(**kw):
    a = tv.PrefillArgs()
    a.struct_size = ctypes.sizeof(tv.PrefillArgs)
    a.B, a.H, a.T, a.d_latent, a.d_nope, a.d_rope, a.d_v = 2, 16, 100, 512, 128, 64, 128
    a.scale, a.dt = 0.07, tv.TV_BF16
    a.q_nope = a.q_pe = a.w_kv = a.c_kv = a.k_pe = a.q_start = a.prefix_len = a.out = FAKE
    a.ckv_row_stride, a.kpe_row_stride = 512, 64
    a.cache = tv.CacheLayout(FAKE, 64, 10, 0, 6400)
    a.max_q_len, a.max_kv_len, a.total_kv = 64, 640, 1000
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), tv.TV_ERR_INVALID_ARG),
    (dict(B=-1), tv.TV_ERR_INVALID_ARG),
    (dict(H=0), tv.TV_ERR_INVALID_ARG),
    (dict(T=-1), tv.TV_ERR_INVALID_ARG),
    (dict(total_kv=-1), tv.TV_ERR_INVALID_ARG),
    (dict(scale=0.0), tv.TV_ERR_INVALID_ARG),
    (dict(scale=-1.0), tv.TV_ERR_INVALID_ARG),
    (dict(scale=float("nan")), tv.TV_ERR_INVALID_ARG),
    (dict(dt=tv.TV_F32), tv.TV_ERR_UNSUPPORTED),
    (dict(d_nope=64), tv.TV_ERR_UNSUPPORTED),
    (dict(d_rope=32), tv.TV_ERR_UNSUPPORTED),
    (dict(d_v=64), tv.TV_ERR_UNSUPPORTED),
    (dict(d_latent=520, ckv_row_stride=520), tv.TV_ERR_UNSUPPORTED),
    (dict(H=65536), tv.TV_ERR_UNSUPPORTED),
    (dict(B=1 << 19, H=1 << 14), tv.TV_ERR_UNSUPPORTED),
    (dict(total_kv=1 << 31), tv.TV_ERR_UNSUPPORTED),
    (dict(q_nope=None), tv.TV_ERR_INVALID_ARG),
    (dict(q_start=None), tv.TV_ERR_INVALID_ARG),
    (dict(w_kv=FAKE + 8), tv.TV_ERR_INVALID_ARG),
    (dict(out=FAKE + 16), tv.TV_ERR_INVALID_ARG),
    (dict(ckv_row_stride=511), tv.TV_ERR_INVALID_ARG),
    (dict(kpe_row_stride=68), tv.TV_ERR_INVALID_ARG),
    (dict(max_kv_len=641), tv.TV_ERR_INVALID_ARG),
    (dict(cache=tv.CacheLayout(FAKE, 32, 20, 0, 6400)), tv.TV_ERR_UNSUPPORTED),
    (dict(cache=tv.CacheLayout(FAKE, 64, 10, 0, 0)), tv.TV_ERR_INVALID_ARG),
    (dict(cache=tv.CacheLayout(None, 64, 0, 639, 6400)), tv.TV_ERR_INVALID_ARG),
    (dict(cache=tv.CacheLayout(None, 64, 0, 1 << 62, 6400)), tv.TV_ERR_INVALID_ARG),
])
def test_prefill_arguments(tvlib, kw, code):
    lib, a = tv.load(), prefill_args(**kw)
    assert lib.tv_prefill_attn_workspace_size(ctypes.byref(a)) == 0
    assert lib.tv_prefill_attn(ctypes.byref(a), FAKE, 1 << 40, None) == code
    assert lib.tv_last_error()


def test_prefill_workspace(tvlib):
    lib, a = tv.load(), prefill_args()
    need = lib.tv_prefill_attn_workspace_size(ctypes.byref(a))
    assert need >= 1000 * (16 * 512 + 128)
    for ws, size in ((None, need), (FAKE + 64, need), (FAKE, need - 1)):
        assert lib.tv_prefill_attn(ctypes.byref(a), ws, size, None) == tv.TV_ERR_WORKSPACE
    for kw in (dict(B=0), dict(T=0)):
        empty = prefill_args(**kw)
        assert lib.tv_prefill_attn(ctypes.byref(empty), None, 0, None) == tv.TV_OK
