"""The paged dense cache without a GPU: frequencies of rotary positions against their formulas,
the oracle's own pins, and the C ABI's refusals (fake addresses that are never dereferenced:
every check returns before a HIP call)."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from oracle import dense_oracle
from sparse_dictionary_coding_amd import build, fadkv

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(fadkv.LIB_PATH),
                                reason="libfadkv.so not built (run __graft_entry__.build())")

FAKE = 0x7F0000100000          # 256-byte aligned
FAKE2 = 0x7F0000200000
I31 = (1 << 31) - 1


# ---- frequencies ------------------------------------------------------------------------------
@pytest.mark.parametrize("rot,base", [(128, 500000.0), (64, 10000.0), (16, 1e6), (2, 7.5)])
@pytest.mark.parametrize("kw", [
    dict(kind="plain"), dict(kind="linear", factor=8.0),
    dict(kind="bands", factor=8.0, low=1.0, high=4.0, original_len=8192),
    dict(kind="bands", factor=32.0, low=1.0, high=4.0, original_len=8192),
    dict(kind="yarn", factor=4.0, low=1.0, high=32.0, original_len=32768),
    dict(kind="yarn", factor=1.0, low=1.0, high=32.0, original_len=4096)])
def test_rope_freqs_match_their_formulas(rot, base, kw):
    got, m = fadkv.fadkv_rope_freqs(rot, base, device="cpu", **kw)
    ref, mref = dense_oracle.rope_freqs(rot, base, **kw)
    # pow, a product and a sum in 64 bits on both sides
    np.testing.assert_allclose(got.numpy(), ref, rtol=1e-13)
    assert m == pytest.approx(mref, rel=1e-15)
    assert got[0] == (1.0 / kw.get("factor", 1.0) if kw["kind"] == "linear" else got[0])


def test_rope_freqs_bands_keep_short_and_stretch_long_waves():
    f, _ = fadkv.fadkv_rope_freqs(128, 500000.0, device="cpu")
    g, _ = fadkv.fadkv_rope_freqs(128, 500000.0, "bands", 8.0, 1.0, 4.0, 8192, device="cpu")
    w = 2 * math.pi / f
    assert (g[w < 2048] == f[w < 2048]).all()
    assert ((g / f)[w > 8192] - 0.125).abs().max() < 1e-15
    mid = (w > 2048) & (w < 8192)
    assert mid.any() and ((g < f) & (g > f / 8))[mid].all()


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=3), -3), (dict(rot_dim=0), -3), (dict(rot_dim=-2), -3), (dict(base=1.0), -1),
    (dict(base=float("nan")), -1), (dict(kind="linear", factor=0.5), -1),
    (dict(kind="bands", factor=8.0, low=4.0, high=4.0), -1),
    (dict(kind="yarn", factor=8.0, original_len=0), -1),
    (dict(kind="yarn", factor=float("inf")), -1)])
def test_rope_freqs_refusals(kw, status):
    base = dict(rot_dim=64, base=10000.0)
    with pytest.raises(fadkv.FadkvError) as e:
        fadkv.fadkv_rope_freqs(**{**base, **kw}, device="cpu")
    assert e.value.status == status


def test_rope_freqs_unknown_kind():
    with pytest.raises(ValueError):
        fadkv.fadkv_rope_freqs(64, 10000.0, "other", device="cpu")


# ---- the oracle's pins --------------------------------------------------------------------------
def test_oracle_pages_by_hand():
    # 4-token pages; row 0 holds 3 tokens and adds 2 (one new page), row 1 ends, row 2 is empty
    # and adds 5 (two pages), row 3 wants one page more than are left
    out = dense_oracle.pages_advance(
        4, [2, -1, 5, 4], [3, 8, 0, 4], [[9, -1, -1], [1, 2, -1], [-1] * 3, [0, -1, -1]],
        [7, 6, 5, 0, 0, 0, 0, 0, 0, 0], [0, 3], 13)
    assert out["status"].tolist() == [0, 2, 0, 1]
    assert out["table"].tolist() == [[9, 7, -1], [1, 2, -1], [6, 5, -1], [0, -1, -1]]
    assert out["lens"].tolist() == [5, 0, 5, 4]
    assert out["cu"].tolist() == [0, 2, 2, 7, 11]
    assert out["slots"].tolist() == [39, 28, 24, 25, 26, 27, 20] + [-1] * 6
    assert out["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, 4, 5, 6, 7, -1, -1]
    assert out["ring"].tolist()[:5] == [7, 6, 5, 1, 2] and out["ring_state"].tolist() == [3, 2]


def test_oracle_norm_rope_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y, _ = dense_oracle.norm_rope(x, np.ones(4), [1], [math.pi / 2], 0.0, True, 1.0)
    np.testing.assert_allclose(y[0, 0], [-1.6, 1.2, 0, 0], atol=1e-15)   # norm 2.5, quarter turn
    y, _ = dense_oracle.norm_rope(x, None, [2], [math.pi / 2, 0.0], 0.0, False, 2.0)
    np.testing.assert_allclose(y[0, 0], [-6, 8, 0, 0], atol=1e-14)       # pairs (0, 2), (1, 3)


def test_oracle_attention_matches_a_mask_by_hand():
    seen = [t for t in range(12) if dense_oracle.visible(9, t, 3, 2)]
    assert seen == [0, 1, 7, 8, 9]
    assert [t for t in range(5) if dense_oracle.visible(1, t, 0, 0)] == [0, 1]
    o, a, _, _ = dense_oracle.attend_query(np.zeros(2), 9, np.ones((12, 2)), np.eye(12)[:, [0, 8]],
                                           [True] * 12, 1.0, 3, 2)
    np.testing.assert_allclose(o, [0.2, 0.2])


# ---- refusals -----------------------------------------------------------------------------------
def _pages(num_pages=64, page_size=16, kv_heads=8, d=128, dtype=1, k=FAKE, v=FAKE):
    return fadkv.fadkv_pages(num_pages, page_size, kv_heads, d, dtype, k, v)


def _advance(num_pages=64, page_size=16, R=4, max_pages=8, ptr=FAKE, max_tokens=10, ws=FAKE,
             ws_bytes=1 << 30, **at):
    names = ["new_lens", "lens", "table", "ring", "ring_state"]
    outs = ["lens_out", "ring_state_out", "cu", "status", "slots", "positions"]
    p = {k: at.get(k, ptr) for k in names + outs}
    return fadkv.lib().fadkv_pages_advance(num_pages, page_size, R, max_pages,
                                           *[p[k] for k in names], max_tokens,
                                           *[p[k] for k in outs], ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(page_size=24), -3), (dict(page_size=8), -3), (dict(page_size=512), -3),
    (dict(num_pages=0), -3), (dict(max_pages=0), -3), (dict(R=-1), -3), (dict(R=8193), -3),
    (dict(max_tokens=-1), -3), (dict(num_pages=1 << 27), -3), (dict(max_pages=1 << 27), -3),
    (dict(max_tokens=I31 - 100), -3), (dict(R=8192, max_pages=1 << 18), -3),
    *[({k: None}, -1) for k in ("new_lens", "lens", "table", "ring", "ring_state", "lens_out",
                                "ring_state_out", "cu", "status", "slots", "positions")],
    (dict(table=FAKE + 2), -1), (dict(slots=FAKE + 1), -1),
    (dict(ws=None), -4), (dict(ws_bytes=63), -4), (dict(ws=FAKE + 2), -4)])
def test_pages_advance_refusals(kw, status):
    assert _advance(**kw) == status


def test_pages_workspace():
    out = ctypes.c_size_t(7)
    f = fadkv.lib().fadkv_pages_workspace_bytes
    assert f(4, ctypes.byref(out)) == 0 and out.value == 64
    assert f(0, ctypes.byref(out)) == 0 and out.value == 0
    assert f(8193, ctypes.byref(out)) == -3 and f(-1, ctypes.byref(out)) == -3 and f(4, None) == -1


def _norm_rope(q_out=FAKE, pages=None, slots=None, k_rows=None, v_rows=None, **kw):
    base = dict(n=5, heads=4, kv_heads=2, d=64, dtype=2, q=FAKE + 256, k=FAKE, v=FAKE,
                q_stride=256, k_stride=128, v_stride=128, positions=FAKE, q_weight=None,
                k_weight=None, eps=1e-6, freqs=FAKE, rot_dim=64, interleaved=0, mscale=1.0)
    a = fadkv.fadkv_qkv(**{**base, **kw})
    return fadkv.lib().fadkv_norm_rope(ctypes.byref(a), q_out,
                                       ctypes.byref(pages) if pages else None, slots, k_rows,
                                       v_rows, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), -2), (dict(d=96), -3), (dict(n=-1), -3), (dict(n=(1 << 23) + 1), -3),
    (dict(heads=0), -3), (dict(kv_heads=0), -3), (dict(kv_heads=257), -3), (dict(heads=16385), -3),
    (dict(rot_dim=72), -3), (dict(rot_dim=80), -3), (dict(rot_dim=-16), -3), (dict(interleaved=2), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(mscale=float("inf")), -1),
    (dict(freqs=None), -1), (dict(freqs=FAKE + 4), -1), (dict(q_stride=255), -3),
    (dict(k_stride=64), -3), (dict(v_stride=0), -3), (dict(v_stride=1 << 40), -3),
    (dict(q_stride=257), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(q=FAKE + 8), -1), (dict(positions=None), -1), (dict(positions=FAKE + 2), -1),
    (dict(q_weight=FAKE + 8), -1), (dict(k_weight=FAKE + 2), -1), (dict(q_out=None), -1),
    (dict(q_out=FAKE + 4), -1), (dict(k_rows=FAKE + 8), -1), (dict(v_rows=FAKE + 4), -1),
    (dict(q_out=FAKE + 256, q_stride=264), -1),                  # in place needs packed tokens
    (dict(pages=_pages(kv_heads=2, d=64, dtype=2)), -1),         # pages without slots
    (dict(pages=_pages(kv_heads=2, d=64, dtype=1), slots=FAKE), -2),
    (dict(pages=_pages(kv_heads=3, d=64, dtype=2), slots=FAKE), -3),
    (dict(pages=_pages(kv_heads=2, d=128, dtype=2), slots=FAKE), -3),
    (dict(pages=_pages(kv_heads=2, d=64, dtype=2), slots=FAKE + 2), -1),
    (dict(pages=_pages(kv_heads=2, d=64, dtype=2, v=None), slots=FAKE), -1)])
def test_norm_rope_refusals(kw, status):
    assert _norm_rope(**kw) == status


def test_norm_rope_without_tokens_is_a_no_op():
    assert _norm_rope(n=0, q=None, k=None, v=None, positions=None, q_out=None) == 0


BAD_PAGES = [(dict(dtype=9), -2), (dict(d=32), -3), (dict(num_pages=0), -3), (dict(page_size=48), -3),
             (dict(num_pages=1 << 27), -3), (dict(kv_heads=0), -3), (dict(kv_heads=300), -3),
             (dict(k=None), -1), (dict(v=FAKE + 8), -1)]
BAD_ATTEND = [(dict(heads=12), -3), (dict(heads=0), -3), (dict(heads=8 * 65), -3), (dict(R=-1), -3),
              (dict(R=1 << 20), -3), (dict(max_pages=0), -3), (dict(max_pages=1 << 27), -3),
              (dict(scale=float("nan")), -1), (dict(window=-1), -1), (dict(sinks=-2), -1),
              (dict(table=None), -1), (dict(lens=None), -1), (dict(q=None), -1), (dict(out=None), -1),
              (dict(table=FAKE + 2), -1), (dict(lens=FAKE + 1), -1), (dict(q=FAKE + 8), -1),
              (dict(out=FAKE + 4), -1), (dict(out=FAKE2), -1), (dict(max_pages=(1 << 26) + 1), -3)]


def _paged(pages=None, table=FAKE, max_pages=8, lens=FAKE, R=4, q=FAKE2, heads=32, scale=0.1,
           window=0, sinks=0, max_len=100, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return fadkv.lib().fadkv_attend_paged(ctypes.byref(pages or _pages()), table, max_pages, lens,
                                          R, q, heads, scale, window, sinks, max_len, out, ws,
                                          ws_bytes, None)


def _prompt(pages=None, table=FAKE, max_pages=8, lens=FAKE, cu=FAKE, R=4, q=FAKE2, n=20, heads=32,
            scale=0.1, window=0, sinks=0, max_len=100, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return fadkv.lib().fadkv_attend_prompt(ctypes.byref(pages or _pages()), table, max_pages, lens,
                                           cu, R, q, n, heads, scale, window, sinks, max_len, out,
                                           ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_paged, _prompt])
def test_attention_refusals(call):
    for kw, status in BAD_PAGES:
        assert call(pages=_pages(**kw)) == status, kw
    for kw, status in BAD_ATTEND:
        assert call(**kw) == status, kw
    assert call(R=0, table=None, lens=None, q=None, out=None) == 0


def test_attend_paged_refusals_of_its_own():
    assert _paged(max_len=0) == -3 and _paged(max_len=129) == -3
    out = ctypes.c_size_t(0)
    f = fadkv.lib().fadkv_attend_paged_workspace_bytes
    assert f(ctypes.byref(_pages(k=None, v=None)), 1, 32, 4096, ctypes.byref(out)) == 0
    need = out.value
    assert need > 0 and need % 256 == 0
    one = dict(R=1, max_pages=256, max_len=4096)
    assert _paged(**one, ws_bytes=need - 1) == -4
    assert _paged(**one, ws=None) == -4 and _paged(**one, ws=FAKE + 16) == -4
    assert f(ctypes.byref(_pages()), 1, 32, 0, ctypes.byref(out)) == -3
    assert f(ctypes.byref(_pages()), 1, 31, 10, ctypes.byref(out)) == -3
    assert f(ctypes.byref(_pages()), 1, 32, 10, None) == -1
    # no window needs more than the bytes for its cache: what it sees is at most that, and the bytes for
    # a shorter cache are no more
    for R, kv, group, dtype in ((1, 8, 4, 1), (1, 100, 1, 2), (2, 1, 17, 1), (70, 1, 1, 2), (3, 5, 2, 0)):
        p, last = _pages(num_pages=1 << 14, kv_heads=kv, dtype=dtype), 0
        for max_len in (1, 200, 300, 600, 1100, 2000, 2048, 2049, 2100, 4000, 5000, 70000, 131072):
            assert f(ctypes.byref(p), R, kv * group, max_len, ctypes.byref(out)) == 0
            assert out.value >= last
            last = out.value
    # a short cache needs none
    assert f(ctypes.byref(_pages()), 1, 32, 16, ctypes.byref(out)) == 0 and out.value == 0


def test_attend_prompt_refusals_of_its_own():
    assert _prompt(n=-1) == -3 and _prompt(n=(1 << 23) + 1) == -3
    assert _prompt(cu=None) == -1 and _prompt(cu=FAKE + 2) == -1
    assert _prompt(n=0, q=None, out=None) == 0
    assert _prompt(max_len=0) == -3 and _prompt(max_len=129) == -3
    out = ctypes.c_size_t(0)
    f = fadkv.lib().fadkv_attend_prompt_workspace_bytes
    assert f(ctypes.byref(_pages(k=None, v=None)), 1, 20, 32, 4096, ctypes.byref(out)) == 0
    need = out.value
    assert need > 0 and need % 256 == 0
    long = dict(R=1, max_pages=256, max_len=4096)
    assert _prompt(**long, ws_bytes=need - 1) == -4
    assert _prompt(**long, ws=None) == -4 and _prompt(**long, ws=FAKE + 16) == -4
    assert f(ctypes.byref(_pages()), 1, 20, 32, 0, ctypes.byref(out)) == -3
    assert f(ctypes.byref(_pages()), 1, 20, 31, 10, ctypes.byref(out)) == -3
    assert f(ctypes.byref(_pages()), 1, -1, 32, 10, ctypes.byref(out)) == -3
    assert f(ctypes.byref(_pages()), 1, 20, 32, 10, None) == -1
    # enough queries need no split, nor does a short cache
    assert f(ctypes.byref(_pages()), 1, 4096, 32, 1 << 20, ctypes.byref(out)) == 0 and out.value == 0
    assert f(ctypes.byref(_pages()), 1, 20, 32, 256, ctypes.byref(out)) == 0 and out.value == 0


# ---- generated code -----------------------------------------------------------------------------
@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_prompt_kernels_use_m0_for_their_copies_alone(tmp_path):
    """The prompt attention writes M0 in assembly for its copies into LDS, which is sound while the
    compiler keeps nothing there; and no kernel of the dense cache has packed fp32 arithmetic."""
    for name in ("attend_prompt.hip", "attend_paged.hip", "norm_rope.hip", "pages.hip"):
        out = tmp_path / (name + ".s")
        cmd = [HIPCC, *build.HIPCC_FLAGS, f"-I{build.INCLUDE}", f"-I{build.CSRC}",
               "--cuda-device-only", "-S", os.path.join(build.CSRC, name), "-o", str(out)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        lines = [ln.strip() for ln in out.read_text().splitlines()]
        assert not [ln for ln in lines if re.match(r"v_pk_(add|mul|fma)_f32", ln)]
        assert not [ln for ln in lines if re.match(r"scratch_(load|store)", ln)], name
        if name != "attend_prompt.hip":
            continue
        copies = 0
        for i, ln in enumerate(lines):
            if ln.startswith(";") or not re.search(r"\bm0\b", ln):
                continue
            assert re.fullmatch(r"s_mov_b32 m0, s\d+", ln), f"unexpected M0 use: {ln}"
            assert lines[i + 1] == "s_nop 0", lines[i + 1]
            assert lines[i + 2].startswith("global_load_lds_dwordx4 "), lines[i + 2]
            copies += 1
        assert copies > 0


def test_rope_freqs_number_past_32_bits_is_refused():
    with pytest.raises(fadkv.FadkvError):
        fadkv.fadkv_rope_freqs(2 ** 32 + 64, 10000.0, device="cpu")
