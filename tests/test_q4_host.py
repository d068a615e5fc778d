"""The 4-bit cache without a GPU: the oracle's rows against hand-worked ones and
the format's error bound, and what the entry points refuse."""
import ctypes

import numpy as np
import pytest

import paged_kv_gqa_08_gb300 as pa
from oracle import q4_cache as q4
from paged_kv_gqa_08_gb300 import build


def test_codes_and_parameters_of_a_worked_group():
    # 32 values 0, 0.5, 1, ..., 15.5: s = float16(15.5 / 15), c = float16(-16 s)
    x = (np.arange(32, dtype=np.float32) / 2).reshape(1, 1, 32)
    x = np.concatenate([x, np.full((1, 1, 32), 3.0, np.float32)], -1)  # a constant group: s = 0, c = the constant
    u, s, c = q4.quantise(x, 32)
    assert s[0, 0, 0] == np.float16(15.5 / 15) and c[0, 0, 0] == np.float16(-16 * np.float32(np.float16(15.5 / 15)))
    assert s[0, 0, 1] == 0 and c[0, 0, 1] == 3
    assert u[0, 0, 0] == 0 and u[0, 0, 31] == 15 and (np.diff(u[0, 0, :32].astype(int)) >= 0).all()
    assert (u[0, 0, 32:] == 0).all()
    assert np.array_equal(q4.values(u, s, c, 32)[0, 0, 32:], np.full(32, 3.0))


def test_bytes_of_a_worked_row():
    # dims 0..3 with codes 1, 2, 4, 8 -> 1<<6 | (2&3)<<14 | 2>>2 | 4<<2 | 8<<10
    u = np.zeros((1, 1, 64), np.uint8)
    u[0, 0, :4] = (1, 2, 4, 8)
    s = np.full((1, 1, 2), 1.0, np.float16)
    c = np.full((1, 1, 2), -16.0, np.float16)
    row = q4.pack_rows(u, s, c, [0])
    assert row.shape == (1, 48)                       # 32 of codes, 8 of parameters padded to 16
    assert int(row[0, 0]) | int(row[0, 1]) << 8 == (1 << 6) | (2 << 14) | (4 << 2) | (8 << 10)
    assert list(row[0, 32:36]) == [0x00, 0x3C, 0x00, 0xCC]   # 1.0, -16.0
    odd = q4.pack_rows(u, s, c, [1])                  # two pieces of codes: exchanged in odd slots
    assert np.array_equal(odd[0, 16:32], row[0, :16]) and np.array_equal(odd[0, 32:], row[0, 32:])


@pytest.mark.parametrize("hkv,hd,gs", [(1, 64, 64), (1, 64, 32), (2, 64, 32), (8, 128, 32), (4, 128, 64), (8, 128, 128)])
def test_rows_round_trip_and_the_error_bound(hkv, hd, gs):
    rng = np.random.default_rng(hkv * hd + gs)
    x = (rng.standard_normal((33, hkv, hd)) * np.exp(rng.uniform(-6, 6, (33, hkv, 1)))).astype(np.float32)
    slots = rng.permutation(64)[:33]
    u, s, c = q4.quantise(x, gs)
    rows = q4.pack_rows(u, s, c, slots)
    assert rows.shape[1] == q4.row_bytes(hkv, hd, gs)
    for a, b in zip(q4.unpack_rows(rows, slots, hkv, hd, gs), (u, s, c)):
        assert np.array_equal(a, b)
    err = np.abs(q4.values(u, s, c, gs) - x)
    sf, cf = (np.repeat(v.astype(np.float64), gs, -1) for v in (s, c))
    # half a step inside the range; at its ends s and c, each rounded by at most half a float16 unit (2^-11 of the
    # value, 2^-25 among subnormals), may leave the extreme values outside by up to 31 roundings of s and one of c
    bound = sf / 2 + (31 * sf + np.abs(cf)) * 2.0 ** -11 + 32 * 2.0 ** -25 + np.abs(x) * 2.0 ** -22
    assert (err <= bound).all()


def test_non_finite_groups_and_large_values():
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, 5], x[0, 0, 40], x[0, 0, 70], x[0, 0, 100] = np.nan, np.inf, 3e38, -1e9
    u, s, c = q4.quantise(x, 32)
    v = q4.values(u, s, c, 32)[0, 0]
    assert np.isnan(v[:64]).all() and np.isfinite(v[64:]).all()
    assert abs(v[70] - 16384) <= 16 and abs(v[100] + 16384) <= 16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pa.load_library()


FAKE = 1 << 20          # a 16-byte aligned non-null "pointer"; never dereferenced on these paths


def _desc(**kw):
    d = dict(num_q_heads=16, num_kv_heads=8, head_dim=128, page_size=16, num_pages=64, dtype=pa.PA_BF16)
    d.update(kw)
    return pa.CacheDesc(*(d[k] for k in ("num_q_heads", "num_kv_heads", "head_dim", "page_size", "num_pages", "dtype")))


def test_row_bytes(lib):
    assert pa.pa_q4_row_bytes(_desc(), 32) == 640
    assert pa.pa_q4_row_bytes(_desc(), 64) == 576
    assert pa.pa_q4_row_bytes(_desc(), 128) == 544
    assert pa.pa_q4_row_bytes(_desc(num_kv_heads=1, num_q_heads=1, head_dim=64), 64) == 48
    for gs in (0, 16, 48, 256, -32):
        assert pa.pa_q4_row_bytes(_desc(), gs) == 0
    assert pa.pa_q4_row_bytes(_desc(head_dim=64), 128) == 0
    assert pa.pa_q4_row_bytes(_desc(dtype=7), 32) == 0
    for hkv in (1, 2, 4, 8):
        for hd in (64, 128):
            for gs in (32, 64, 128):
                if gs <= hd:
                    assert pa.pa_q4_row_bytes(_desc(num_q_heads=hkv, num_kv_heads=hkv, head_dim=hd),
                                              gs) == q4.row_bytes(hkv, hd, gs)


def _write(lib, desc=None, gs=32, **kw):
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, n=3, slots=FAKE, kc=FAKE, vc=FAKE)
    a.update(kw)
    return lib.pa_kv_write_q4(ctypes.byref(desc or _desc()), gs, a["k"], a["ks"], a["v"], a["vs"], a["n"], a["slots"],
                              a["kc"], a["vc"], None)


def _read(lib, desc=None, gs=32, **kw):
    a = dict(batch=2, cu=FAKE, starts=None, ctx=FAKE, bt=FAKE, maxp=4, rows=5, kc=FAKE, vc=FAKE, ko=FAKE, ks=1024,
             vo=FAKE, vs=1024)
    a.update(kw)
    return lib.pa_kv_read_q4(ctypes.byref(desc or _desc()), gs, a["batch"], a["cu"], a["starts"], a["ctx"], a["bt"],
                             a["maxp"], a["rows"], a["kc"], a["vc"], a["ko"], a["ks"], a["vo"], a["vs"], None)


def _decode(lib, desc=None, gs=32, **kw):
    a = dict(q=FAKE, batch=4, kc=FAKE, vc=FAKE, bt=FAKE, maxp=8, ctx=FAKE, max_ctx=100, scale=0.1, max_ctas=0,
             out=FAKE, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return lib.pa_decode_q4(ctypes.byref(desc or _desc()), gs, a["q"], a["batch"], a["kc"], a["vc"], a["bt"],
                            a["maxp"], a["ctx"], a["max_ctx"], a["scale"], a["max_ctas"], a["out"], a["ws"],
                            a["ws_bytes"], None)


def _step(lib, desc=None, gs=32, **kw):
    a = dict(q=FAKE, kn=FAKE, ks=1024, vn=FAKE, vs=1024, batch=4, kc=FAKE, vc=FAKE, bt=FAKE, maxp=8, ctx=FAKE,
             max_ctx=100, scale=0.1, max_ctas=0, slots=None, out=FAKE, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return lib.pa_decode_kv_write_q4(ctypes.byref(desc or _desc()), gs, a["q"], a["kn"], a["ks"], a["vn"], a["vs"],
                                     a["batch"], a["kc"], a["vc"], a["bt"], a["maxp"], a["ctx"], a["max_ctx"],
                                     a["scale"], a["max_ctas"], a["slots"], a["out"], a["ws"], a["ws_bytes"], None)


def _norm(lib, desc=None, gs=32, **kw):
    a = dict(q=FAKE, qs=2048, k=FAKE, ks=1024, v=FAKE, vs=1024, n=3, pos=FAKE, wq=FAKE, wk=FAKE, eps=1e-6, theta=1e6,
             slots=FAKE, qo=FAKE + 4096, kc=FAKE, vc=FAKE)
    a.update(kw)
    return lib.pa_qk_norm_rope_kv_write_q4(ctypes.byref(desc or _desc()), gs, a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                           a["vs"], a["n"], a["pos"], a["wq"], a["wk"], a["eps"], a["theta"],
                                           a["slots"], a["qo"], a["kc"], a["vc"], None)


def _pnorm(lib, desc=None, gs=32, **kw):
    a = dict(q=FAKE, qs=2048, k=FAKE, ks=1024, v=FAKE, vs=1024, n=3, cu=FAKE, batch=2, ctx=FAKE, bt=FAKE, maxp=4,
             wq=FAKE, wk=FAKE, eps=1e-6, theta=1e6, qo=FAKE + 4096, kc=FAKE, vc=FAKE)
    a.update(kw)
    return lib.pa_prefill_qk_norm_rope_kv_write_q4(
        ctypes.byref(desc or _desc()), gs, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["n"], a["cu"],
        a["batch"], a["ctx"], a["bt"], a["maxp"], a["wq"], a["wk"], a["eps"], a["theta"], a["qo"], a["kc"], a["vc"],
        None, None, None)


@pytest.mark.parametrize("call", [_write, _read, _decode, _step, _norm, _pnorm])
def test_every_call_refuses_a_group_size_it_does_not_have(lib, call):
    for gs in (0, -1, 16, 33, 96, 256):
        assert call(lib, gs=gs) == pa.PA_ERR_UNSUPPORTED
    assert call(lib, _desc(head_dim=64), gs=128) == pa.PA_ERR_UNSUPPORTED
    assert call(lib, _desc(dtype=3)) == pa.PA_ERR_DTYPE
    assert call(lib, _desc(num_kv_heads=3, num_q_heads=3)) == pa.PA_ERR_UNSUPPORTED
    assert call(lib, _desc(num_q_heads=72)) == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,bad", [
    (_write, dict(k=None)), (_write, dict(v=None)), (_write, dict(slots=None)), (_write, dict(kc=None)),
    (_read, dict(cu=None)), (_read, dict(ctx=None)), (_read, dict(bt=None)), (_read, dict(ko=None)),
    (_read, dict(vc=None)), (_decode, dict(q=None)), (_decode, dict(kc=None)), (_decode, dict(out=None)),
    (_step, dict(kn=None)), (_step, dict(vn=None)), (_step, dict(ctx=None)), (_norm, dict(pos=None)),
    (_norm, dict(slots=None)), (_norm, dict(wk=None)), (_norm, dict(qo=None)), (_pnorm, dict(cu=None)),
    (_pnorm, dict(bt=None))])
def test_null_pointers(lib, call, bad):
    assert call(lib, **bad) == pa.PA_ERR_NULL


@pytest.mark.parametrize("call,bad,status", [
    (_write, dict(ks=1016), pa.PA_ERR_SHAPE), (_write, dict(vs=1028), pa.PA_ERR_ALIGN),
    (_write, dict(n=-1), pa.PA_ERR_SHAPE), (_write, dict(kc=FAKE + 8), pa.PA_ERR_ALIGN),
    (_write, dict(k=FAKE + 2), pa.PA_ERR_ALIGN),
    (_read, dict(rows=-1), pa.PA_ERR_SHAPE), (_read, dict(batch=0), pa.PA_ERR_SHAPE),
    (_read, dict(batch=-1), pa.PA_ERR_SHAPE), (_read, dict(maxp=0), pa.PA_ERR_SHAPE),
    (_read, dict(ks=1000), pa.PA_ERR_SHAPE), (_read, dict(vs=1025), pa.PA_ERR_ALIGN),
    (_read, dict(vo=FAKE + 4), pa.PA_ERR_ALIGN), (_read, dict(rows=1 << 31), pa.PA_ERR_SHAPE),
    (_decode, dict(batch=-1), pa.PA_ERR_SHAPE), (_decode, dict(max_ctx=129), pa.PA_ERR_SHAPE),
    (_decode, dict(max_ctas=-1), pa.PA_ERR_SHAPE), (_decode, dict(scale=float("nan")), pa.PA_ERR_SHAPE),
    (_decode, dict(ws=None), pa.PA_ERR_WORKSPACE), (_decode, dict(ws=FAKE + 16), pa.PA_ERR_ALIGN),
    (_step, dict(ks=1016), pa.PA_ERR_SHAPE), (_step, dict(vn=FAKE + 8), pa.PA_ERR_ALIGN),
    (_step, dict(ws=None), pa.PA_ERR_WORKSPACE),
    (_norm, dict(qs=2040), pa.PA_ERR_SHAPE), (_norm, dict(eps=-1.0), pa.PA_ERR_SHAPE),
    (_norm, dict(theta=1.0), pa.PA_ERR_SHAPE), (_pnorm, dict(batch=0), pa.PA_ERR_SHAPE),
    (_pnorm, dict(maxp=0), pa.PA_ERR_SHAPE)])
def test_bad_sizes_and_alignment(lib, call, bad, status):
    assert call(lib, **bad) == status


def test_the_fused_step_refuses_slots_past_32_bits(lib):
    assert _step(lib, _desc(num_pages=1 << 27)) == pa.PA_ERR_UNSUPPORTED


def test_empty_calls_do_nothing(lib):
    assert _write(lib, n=0) == pa.PA_OK
    assert _norm(lib, n=0) == pa.PA_OK
    assert _pnorm(lib, n=0) == pa.PA_OK
    assert _read(lib, rows=0) == pa.PA_OK
    assert _decode(lib, batch=0) == pa.PA_OK
    assert _step(lib, batch=0) == pa.PA_OK


def test_the_binding_refuses_caches_that_are_not_4_bit_rows():
    torch = pytest.importorskip("torch")
    desc = _desc(num_pages=2)
    good = torch.zeros(2 * 16, 640, dtype=torch.uint8)
    for bad, status in ((torch.zeros(2, 16, 8, 128, dtype=torch.bfloat16), pa.PA_ERR_DTYPE),
                        (torch.zeros(2 * 16, 639, dtype=torch.uint8), pa.PA_ERR_SHAPE),
                        (torch.zeros(2 * 16, 1280, dtype=torch.uint8)[:, ::2], pa.PA_ERR_SHAPE),
                        (good, pa.PA_ERR_UNSUPPORTED)):   # host memory
        with pytest.raises(pa.PagedAttnError) as e:
            pa.pa_kv_write_q4(desc, 32, FAKE, 1024, FAKE, 1024, 1, FAKE, bad, bad)
        assert e.value.status == status


@pytest.fixture
def enqueued(monkeypatch):
    """The calls of the library that a step makes, recorded in place of made: these tests need no GPU and touch none."""
    from paged_kv_gqa_08_gb300 import step
    calls = []
    for name in [n for n in vars(step) if n.startswith("pa_") and not n.endswith("workspace_size")]:
        monkeypatch.setattr(step, name, lambda *a, name=name, **k: calls.append(name))
    monkeypatch.setattr(step, "pa_decode_q4_workspace_size", lambda *a: 4096)
    monkeypatch.setattr(step, "pa_prefill_workspace_size", lambda *a: 4096)
    return calls


def _step_args(kind="prefill", **kw):
    """Buffers and arguments of run_step over a 4-bit cache of two requests, in host memory."""
    import torch
    from paged_kv_gqa_08_gb300.step import alloc_step_buffers

    desc = _desc(num_pages=8)
    bufs = alloc_step_buffers(desc, kind, 6, 2, 64, "cpu", norm=True, max_seqlen_q=8, group_size=32)
    base = torch.zeros(8192, dtype=torch.uint8)
    at = -base.data_ptr() % 256
    bufs.workspace = base[at: at + 4096]
    n = 6 if kind == "prefill" else 2
    cache = torch.zeros(8 * 16, 640, dtype=torch.uint8)
    rows = torch.zeros(n, 8, 128, dtype=torch.bfloat16)
    a = dict(desc=desc, kind=kind, bufs=bufs, q=torch.zeros(n, 16, 128, dtype=torch.bfloat16), k=rows, v=rows,
             cu_seqlens_q=torch.tensor([0, n // 2, n], dtype=torch.int32),
             context_lens=torch.tensor([20, 30], dtype=torch.int32),
             block_tables=torch.zeros(2, 4, dtype=torch.int32), k_cache=cache, v_cache=cache, scale=0.1,
             max_pages_per_seq=4, max_context_len=64, max_seqlen_q=8, q_norm_w=None, k_norm_w=None, eps=1e-6,
             rope_theta=1e4)
    a.update(kw)
    return a


def _wide(torch, a):             # q's rows inside a fused projection
    a["q"] = torch.zeros(a["q"].shape[0], 32, 128, dtype=torch.bfloat16)[:, :16]


def _transposed(torch, a):
    a["q"] = torch.zeros(a["q"].shape[0], 128, 16, dtype=torch.bfloat16).transpose(1, 2)


def _past_the_tables(torch, a):
    a["max_context_len"] = 65
    if a["bufs"].staging is not None:
        a["bufs"].staging.max_pages = 5


def _misaligned(torch, like):
    return torch.zeros(like.numel() + 8, dtype=like.dtype)[1: 1 + like.numel()].view(like.shape)


def _small_workspace(torch, a):
    a["bufs"].workspace = a["bufs"].workspace[:4095]


def _odd_workspace(torch, a):
    base = torch.zeros(8192, dtype=torch.uint8)
    a["bufs"].workspace = base[16 - base.data_ptr() % 256 + 256:]


@pytest.mark.parametrize("kind", ["prefill", "decode"])
@pytest.mark.parametrize("spoil,status", [
    (lambda torch, a: a.update(q_norm_w=torch.ones(128, dtype=torch.bfloat16)), pa.PA_ERR_NULL),
    (lambda torch, a: a.update(k_norm_w=torch.ones(128, dtype=torch.bfloat16)), pa.PA_ERR_NULL),
    (_wide, pa.PA_ERR_SHAPE), (_transposed, pa.PA_ERR_SHAPE), (_past_the_tables, pa.PA_ERR_SHAPE),
    (lambda torch, a: a.update(max_context_len=0), pa.PA_ERR_SHAPE),
    (lambda torch, a: a.update(scale=float("nan")), pa.PA_ERR_SHAPE),
    (lambda torch, a: a.update(q=_misaligned(torch, a["q"])), pa.PA_ERR_ALIGN),
    (lambda torch, a: setattr(a["bufs"], "out", _misaligned(torch, a["bufs"].out)), pa.PA_ERR_ALIGN),
    (_small_workspace, pa.PA_ERR_WORKSPACE), (_odd_workspace, pa.PA_ERR_ALIGN)])
def test_a_step_is_refused_before_anything_is_enqueued(enqueued, kind, spoil, status):
    torch = pytest.importorskip("torch")
    from paged_kv_gqa_08_gb300.step import run_step

    a = _step_args(kind)
    spoil(torch, a)
    with pytest.raises(pa.PagedAttnError) as e:
        run_step(**a)
    assert e.value.status == status and not enqueued


@pytest.mark.parametrize("spoil,status", [
    (lambda torch, a: a.update(q_norm_w=torch.ones(128, dtype=torch.bfloat16)), pa.PA_ERR_NULL),
    (lambda torch, a: a.update(k_norm_w=torch.ones(128, dtype=torch.bfloat16)), pa.PA_ERR_NULL),
    (_wide, pa.PA_ERR_SHAPE), (_transposed, pa.PA_ERR_SHAPE)])
def test_a_decode_step_over_rows_of_the_dtype_looks_at_its_queries_first(enqueued, spoil, status):
    torch = pytest.importorskip("torch")
    from paged_kv_gqa_08_gb300.step import run_step

    a = _step_args("decode")
    a["bufs"].group_size = 0
    spoil(torch, a)
    with pytest.raises(pa.PagedAttnError) as e:
        run_step(**a)
    assert e.value.status == status and not enqueued


@pytest.mark.parametrize("kw,status", [(dict(max_seqlen_q=0), pa.PA_ERR_SHAPE), (dict(max_seqlen_q=65), pa.PA_ERR_SHAPE),
                                       (dict(scale=0.0), pa.PA_ERR_SHAPE), (dict(scale=-1.0), pa.PA_ERR_SHAPE)])
def test_a_prefill_step_is_refused_before_anything_is_enqueued(enqueued, kw, status):
    pytest.importorskip("torch")
    from paged_kv_gqa_08_gb300.step import run_step

    with pytest.raises(pa.PagedAttnError) as e:
        run_step(**_step_args(**kw))
    assert e.value.status == status and not enqueued


def test_a_prefill_step_beyond_its_buffers_is_refused_before_anything_is_enqueued(enqueued):
    pytest.importorskip("torch")
    from paged_kv_gqa_08_gb300.step import run_step

    decode_bufs = _step_args()
    decode_bufs["bufs"].staging = None
    for a in (_step_args(max_context_len=65, max_pages_per_seq=5), decode_bufs):
        with pytest.raises(ValueError):
            run_step(**a)
        assert not enqueued


@pytest.mark.parametrize("kind", ["prefill", "decode"])
@pytest.mark.parametrize("group_size", [32, 0])
@pytest.mark.parametrize("short", ["positions", "slots", "out", "q_out"])
def test_a_step_of_more_tokens_than_its_buffers_hold_is_refused(enqueued, kind, group_size, short):
    torch = pytest.importorskip("torch")
    from paged_kv_gqa_08_gb300.step import run_step

    w = torch.ones(128, dtype=torch.bfloat16)
    a = _step_args(kind, q_norm_w=w, k_norm_w=w)
    bufs = a["bufs"]
    bufs.group_size = group_size
    setattr(bufs, short, getattr(bufs, short)[: a["q"].shape[0] - 1])
    with pytest.raises(ValueError):
        run_step(**a)
    assert not enqueued


def test_steps_that_are_not_refused(enqueued):
    torch = pytest.importorskip("torch")
    from paged_kv_gqa_08_gb300.step import run_step

    w = torch.ones(128, dtype=torch.bfloat16)
    run_step(**_step_args())
    run_step(**_step_args("decode"))
    assert enqueued[-1] == "pa_decode_q4"
    wide = torch.zeros(6, 32, 128, dtype=torch.bfloat16)[:, :16]
    run_step(**_step_args(q=wide, q_norm_w=w, k_norm_w=w))          # the norm takes rows of any stride
    run_step(**_step_args(q=wide[:1], cu_seqlens_q=torch.tensor([0, 0, 1], dtype=torch.int32)))   # one row has none
    run_step(**_step_args("decode", scale=-0.1))
    a = _step_args()
    a["bufs"].workspace = None                                      # prefill takes none, too
    run_step(**a)
    assert enqueued.count("pa_prefill_varlen") == 4 and enqueued.count("pa_decode_q4") == 2


def test_read_back_tables_refusals(lib):
    def call(desc=None, batch=2, cu=FAKE, bt=FAKE, maxp=4, out=FAKE, maxp_out=4):
        return lib.pa_kv_read_q4_tables(ctypes.byref(desc or _desc()), batch, cu, bt, maxp, out, maxp_out, None)

    assert call(batch=0) == pa.PA_OK
    assert call(desc=_desc(dtype=7)) == pa.PA_ERR_DTYPE
    assert call(desc=_desc(page_size=24)) == pa.PA_ERR_UNSUPPORTED
    for bad in (dict(batch=-1), dict(maxp=0), dict(maxp_out=0), dict(batch=1 << 20, maxp_out=1 << 20)):
        assert call(**bad) == pa.PA_ERR_SHAPE
    for bad in (dict(cu=None), dict(bt=None), dict(out=None)):
        assert call(**bad) == pa.PA_ERR_NULL
