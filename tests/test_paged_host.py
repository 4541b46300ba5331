"""Refusals of the paged-cache entry points, on the host before any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from scaled_dot_product_04_gb300 import _lib
    return _lib.load()


def _status(L, rc, text=""):
    return rc, text in L.sdpa_last_error()


def _plan(lib, ctx=0x1000, new=0x2000, parents=0x3000, held=0x4000, state=0x5000, ring=0x6000,
          table=0x10000, held_out=0x7000, state_out=0x8000, cu=0x9000, kv=0xa000, slots=0xb000,
          pos=0xc000, mask=0xd000, b=4, blocks=8, page=16, pages=32, max_new=20, words=1):
    return lib.sdpa_cache_plan(ctx, new, parents, held, state, ring, table, held_out, state_out, cu,
                               kv, slots, pos, mask, b, blocks, page, pages, max_new, words, None)


def test_plan_refusals(lib):
    from scaled_dot_product_04_gb300 import _lib as L
    for kw, status, text in [
            (dict(page=24), L.SDPA_ERR_UNSUPPORTED, "page_size 24"),
            (dict(page=8), L.SDPA_ERR_UNSUPPORTED, "page_size 8"),
            (dict(page=192), L.SDPA_ERR_UNSUPPORTED, "page_size 192"),
            (dict(b=-1), L.SDPA_ERR_INVALID_ARG, "negative"),
            (dict(max_new=-1), L.SDPA_ERR_INVALID_ARG, "negative"),
            (dict(pages=0), L.SDPA_ERR_INVALID_ARG, "num_pages is 0"),
            (dict(pages=1 << 28), L.SDPA_ERR_INVALID_ARG, "31 bits"),
            (dict(parents=None), L.SDPA_ERR_INVALID_ARG, "needs parents"),
            (dict(words=0), L.SDPA_ERR_INVALID_ARG, "mask_words"),
            (dict(mask=None), L.SDPA_ERR_INVALID_ARG, "without tree_mask"),
            (dict(b=0), L.SDPA_ERR_INVALID_ARG, "num_seqs is 0"),
            (dict(ctx=None), L.SDPA_ERR_INVALID_ARG, "ctx_lens is NULL"),
            (dict(slots=0xb002), L.SDPA_ERR_MISALIGNED, "slot_map"),
            (dict(held_out=0x4000), L.SDPA_ERR_INVALID_ARG, "overlaps"),
            (dict(state_out=0x5004), L.SDPA_ERR_INVALID_ARG, "overlaps"),
            (dict(b=1 << 20, blocks=1 << 12), L.SDPA_ERR_INVALID_ARG, "too large"),
            (dict(max_new=(1 << 30) + 1), L.SDPA_ERR_INVALID_ARG, "too large")]:
        assert _plan(lib, **kw) == status, (kw, L.sdpa_last_error())
        assert text in L.sdpa_last_error(), (kw, L.sdpa_last_error())


def _append(lib, k=0x100000, v=0x200000, kc=0x300000, vc=0x400000, slots=0x500000, sk=0x600000,
            sv=0x600010, total=10, ks=1024, vs=1024, h_kv=8, d=128, pages=4, page=16, dtype=0, cache=0):
    return lib.sdpa_cache_append(k, v, kc, vc, slots, sk, sv, total, ks, vs, h_kv, d, pages, page,
                                 dtype, cache, None)


def test_append_refusals(lib):
    from scaled_dot_product_04_gb300 import _lib as L
    for kw, status, text in [
            (dict(d=96), L.SDPA_ERR_UNSUPPORTED, "d=96"),
            (dict(dtype=2), L.SDPA_ERR_UNSUPPORTED, "dtype 2"),
            (dict(cache=1), L.SDPA_ERR_UNSUPPORTED, "cache_dtype 1"),
            (dict(cache=2, d=64), L.SDPA_ERR_UNSUPPORTED, "d = 128"),
            (dict(cache=2, sk=None), L.SDPA_ERR_INVALID_ARG, "scale_k"),
            (dict(ks=1000), L.SDPA_ERR_INVALID_ARG, "k_stride"),
            (dict(vs=1028), L.SDPA_ERR_INVALID_ARG, "v_stride"),
            (dict(total=-1), L.SDPA_ERR_INVALID_ARG, "negative"),
            (dict(kc=0x300008), L.SDPA_ERR_MISALIGNED, "k_cache"),
            (dict(vc=0x300000), L.SDPA_ERR_INVALID_ARG, "overlap"),
            (dict(kc=0x100000), L.SDPA_ERR_INVALID_ARG, "overlaps input k")]:
        assert _append(lib, **kw) == status, (kw, L.sdpa_last_error())
        assert text in L.sdpa_last_error(), (kw, L.sdpa_last_error())
    assert _append(lib, total=0) == L.SDPA_OK


def _accept(lib, kc=0x300000, vc=0x400000, table=0x1000, ctx=0x2000, new=0x3000, path=0x4000,
            plen=0x5000, out=0x6000, b=4, blocks=8, max_path=5, h_kv=8, d=128, pages=4, page=16, cache=0):
    return lib.sdpa_cache_accept(kc, vc, table, ctx, new, path, plen, out, b, blocks, max_path, h_kv,
                                 d, pages, page, cache, None)


def test_accept_refusals(lib):
    from scaled_dot_product_04_gb300 import _lib as L
    for kw, status, text in [
            (dict(cache=3), L.SDPA_ERR_UNSUPPORTED, "dtype 3"),
            (dict(page=48), L.SDPA_ERR_UNSUPPORTED, "page_size 48"),
            (dict(max_path=-1), L.SDPA_ERR_INVALID_ARG, "negative"),
            (dict(out=0x2000), L.SDPA_ERR_INVALID_ARG, "overlaps"),
            (dict(path=None), L.SDPA_ERR_INVALID_ARG, "path is NULL")]:
        assert _accept(lib, **kw) == status, (kw, L.sdpa_last_error())
        assert text in L.sdpa_last_error(), (kw, L.sdpa_last_error())
    assert _accept(lib, b=0) == L.SDPA_OK


def _tree(lib, q=0x1000000, kc=0x2000000, vc=0x3000000, o=0x4000000, lse=None, table=0x1000, cu=0x2000,
          kv=0x3000, mask=0x4000, dk=0x5000, dv=0x5010, b=2, total=10, mq=6, mkv=100, blocks=8, words=1,
          qs=None, h=8, h_kv=2, d=128, pages=16, page=16, scale=0.1, dtype=0, cache=0, ws=0x8000000,
          ws_bytes=1 << 40):
    return lib.sdpa_tree_fwd(q, kc, vc, o, lse, table, cu, kv, mask, dk, dv, b, total, mq, mkv, blocks,
                             words, h * d if qs is None else qs, h, h_kv, d, pages, page, scale, dtype,
                             cache, ws, ws_bytes, None)


def test_tree_refusals(lib):
    from scaled_dot_product_04_gb300 import _lib as L
    for kw, status, text in [
            (dict(d=32), L.SDPA_ERR_UNSUPPORTED, "d=32"),
            (dict(h_kv=3), L.SDPA_ERR_INVALID_ARG, "multiple of h_kv"),
            (dict(h=129, h_kv=1), L.SDPA_ERR_UNSUPPORTED, "128 query heads"),
            (dict(scale=0.0), L.SDPA_ERR_INVALID_ARG, "attn_scale"),
            (dict(cache=2, dv=None), L.SDPA_ERR_INVALID_ARG, "descale_v"),
            (dict(words=0), L.SDPA_ERR_INVALID_ARG, "mask_words"),
            (dict(mq=11), L.SDPA_ERR_INVALID_ARG, "exceeds total_q"),
            (dict(mq=0), L.SDPA_ERR_INVALID_ARG, "max_seqlen_q is 0"),
            (dict(b=0), L.SDPA_ERR_INVALID_ARG, "num_seqs 0"),
            (dict(qs=1020), L.SDPA_ERR_INVALID_ARG, "q_stride"),
            (dict(qs=1000), L.SDPA_ERR_INVALID_ARG, "q_stride"),
            (dict(o=0x1000000), L.SDPA_ERR_INVALID_ARG, "overlaps input q"),
            (dict(kv=0x3001), L.SDPA_ERR_MISALIGNED, "kv_lens"),
            (dict(table=None), L.SDPA_ERR_INVALID_ARG, "block_table is NULL"),
            (dict(b=1 << 20, total=1 << 20, mkv=1 << 20), L.SDPA_ERR_INVALID_ARG, "too large"),
            (dict(pages=0), L.SDPA_ERR_INVALID_ARG, "num_pages is 0"),
            (dict(ws_bytes=100), L.SDPA_ERR_WORKSPACE, "workspace has 100"),
            (dict(mkv=-1), L.SDPA_ERR_INVALID_ARG, "negative")]:
        assert _tree(lib, **kw) == status, (kw, L.sdpa_last_error())
        assert text in L.sdpa_last_error(), (kw, L.sdpa_last_error())
    assert _tree(lib, total=0, mq=0) == L.SDPA_OK
    none = ctypes.c_size_t(-1).value
    assert L.sdpa_tree_fwd_workspace_size(1, 1, 1, 4, 3, 128) == none
    assert L.sdpa_tree_fwd_workspace_size(1, 1, 1, 4, 4, 96) == none
    assert L.sdpa_tree_fwd_workspace_size(-1, 1, 1, 4, 4, 64) == none
    assert 0 <= L.sdpa_tree_fwd_workspace_size(4, 8, 1000, 8, 2, 128) < 1 << 30


def test_python_refuses_what_pointers_cannot_say():
    """Shapes, types and layouts that the C ABI cannot see (CPU tensors: nothing is launched)."""
    import torch

    import scaled_dot_product_04_gb300 as sdpa
    from scaled_dot_product_04_gb300 import _lib as L
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(sdpa.SdpaError) as e:
        sdpa.cache_append(k, k, cache, cache.clone(), slots)
    assert e.value.status == L.SDPA_ERR_INVALID_ARG and "not on the GPU" in str(e.value)
    with pytest.raises(sdpa.SdpaError) as e:
        sdpa.cache_append(k, k, cache.float(), cache.float(), slots)
    assert e.value.status == L.SDPA_ERR_UNSUPPORTED


INT_MAX = 2 ** 31 - 1


def test_tree_bounds_near_32_bits_are_counted_in_64(lib):
    """max_seqlen_kv is any upper bound: the key tiles that it allows are counted without overflow, and a list of
    them past 31 bits is refused; so is a table whose last tile would end past 31 bits."""
    from scaled_dot_product_04_gb300 import _lib as L
    for kw in [dict(b=100, total=100, mq=1, mkv=INT_MAX),
               dict(b=100, total=100, mq=1, mkv=INT_MAX - 100),
               dict(b=4000, total=4000, mq=1, mkv=INT_MAX - 126),
               dict(b=1, mkv=100, blocks=(1 << 27) - 1, page=16),
               dict(b=1, mkv=100, blocks=(1 << 24) - 1, page=128)]:
        assert _tree(lib, **kw) == L.SDPA_ERR_INVALID_ARG, (kw, L.sdpa_last_error())
        assert "too large for one launch" in L.sdpa_last_error(), (kw, L.sdpa_last_error())


def test_plan_refuses_more_requests_than_its_scan_counts(lib):
    """With no table columns, the table's size alone does not bound the requests."""
    from scaled_dot_product_04_gb300 import _lib as L
    for b in ((1 << 30) + 1, INT_MAX):
        assert _plan(lib, b=b, blocks=0) == L.SDPA_ERR_INVALID_ARG, L.sdpa_last_error()
        assert "too large for one launch" in L.sdpa_last_error()


def test_accept_refuses_rows_wider_than_a_grid(lib):
    """A launch has 65,535 CTAs of 128 16-byte columns over the heads of both caches."""
    from scaled_dot_product_04_gb300 import _lib as L
    most = 65535 * 128 // (2 * 16)  # d = 128, 16 bits: 16 columns a row
    for h in (most + 1, 1 << 27):
        assert _accept(lib, h_kv=h, pages=0) == L.SDPA_ERR_INVALID_ARG, L.sdpa_last_error()
        assert "too large for one launch" in L.sdpa_last_error()


def test_first_use_from_two_threads_builds_once(monkeypatch):
    """Two threads' first calls: one build at a time, one module."""
    import threading
    import time

    from scaled_dot_product_04_gb300 import _lib as L
    L.calls()
    running, most, lock = [0], [0], threading.Lock()
    path = L._build.build_calls()

    def build_calls():
        with lock:
            running[0] += 1
            most[0] = max(most[0], running[0])
        time.sleep(0.2)
        with lock:
            running[0] -= 1
        return path

    monkeypatch.setattr(L, "_calls", None)
    monkeypatch.setattr(L._build, "build_calls", build_calls)
    got = []
    threads = [threading.Thread(target=lambda: got.append(L.calls())) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert len(got) == 4 and all(m is got[0] for m in got) and most[0] == 1


def test_compilers_of_two_threads_write_to_different_files(monkeypatch, tmp_path):
    """Whoever builds at the same time as another installs a module that is whole."""
    import threading

    from scaled_dot_product_04_gb300 import build
    calls = tmp_path / "_sdpa_calls.so"
    monkeypatch.setattr(build, "CALLS", str(calls))
    written, meet = [], threading.Barrier(2)

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        written.append(out)
        with open(out, "w") as f:
            f.write("whole")
        meet.wait(30)
        return type("Done", (), {"returncode": 0, "stdout": "", "stderr": ""})()

    monkeypatch.setattr(build.subprocess, "run", run)
    failed = []

    def one():
        try:
            build.build_calls(force=True)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=one) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed and len(set(written)) == 2 and calls.read_text() == "whole"


def test_the_compiled_entry_goes_with_its_python(monkeypatch):
    """A module built for another Python is not taken for an up-to-date one."""
    import sysconfig

    from scaled_dot_product_04_gb300 import build
    build.build_calls()
    assert build.calls_up_to_date()
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other" if name == "SOABI" else real(name))
    assert not build.calls_up_to_date()
