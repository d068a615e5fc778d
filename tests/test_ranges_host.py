"""What the windowed, shared-prefix and block-table calls refuse on the host, without a GPU."""
import ctypes

import pytest

import paged_kv_gqa_08_gb300 as pa
from paged_kv_gqa_08_gb300 import build

FAKE = 0x10000   # an aligned address that no call here reaches


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pa.load_library()


def _desc(**kw):
    d = dict(num_q_heads=16, num_kv_heads=8, head_dim=128, page_size=16, num_pages=64, dtype=pa.PA_BF16)
    d.update(kw)
    return pa.cache_desc(**d)


DECODE = ("q", "batch", "k_cache", "v_cache", "block_tables", "max_pages", "context_lens", "max_context_len", "scale",
          "max_ctas", "out", "workspace", "bytes", "stream")
CALLS = {
    "pa_decode_window": ("desc", "window", "sinks") + DECODE,
    "pa_decode_kv_write_window": ("desc", "window", "sinks", "q", "k", "k_stride", "v", "v_stride", "batch", "k_cache",
                                  "v_cache", "block_tables", "max_pages", "context_lens", "max_context_len", "scale",
                                  "max_ctas", "slots", "out", "workspace", "bytes", "stream"),
    "pa_prefill_varlen_window": ("desc", "window", "sinks", "q", "cu", "batch", "max_seqlen_q", "num_tokens", "k_cache",
                                 "v_cache", "block_tables", "max_pages", "context_lens", "max_context_len", "scale",
                                 "out", "workspace", "bytes", "stream"),
    "pa_decode_shared_prefix": ("desc", "groups", "cu_groups", "prefix_lens", "max_prefix") + DECODE,
    "pa_extend_tables": ("desc", "batch", "new", "context_lens", "block_tables", "max_pages", "ring", "pool",
                         "max_tokens", "cu", "ctx_out", "positions", "slots", "refs", "pool_out", "stream"),
    "pa_share_pages": ("desc", "batch", "parents", "counts", "block_tables", "max_pages", "refs", "stream"),
    "pa_release_pages": ("desc", "batch", "first", "end", "block_tables", "max_pages", "refs", "ring", "pool",
                         "pool_out", "stream"),
    "pa_release_window_pages": ("desc", "window", "sinks", "batch", "context_lens", "block_tables", "max_pages", "refs",
                                "ring", "pool", "pool_out", "stream"),
}
NUMBERS = dict(window=64, sinks=4, batch=2, max_pages=8, max_context_len=128, scale=0.1, max_ctas=0, bytes=1 << 30,
               stream=None, k_stride=1024, v_stride=1024, max_seqlen_q=64, num_tokens=100, groups=2, max_prefix=100,
               max_tokens=10, refs=FAKE)
ATTENTION = ("pa_decode_window", "pa_decode_kv_write_window", "pa_prefill_varlen_window", "pa_decode_shared_prefix")


def call(lib, fn, **kw):
    a = {**{n: FAKE for n in CALLS[fn]}, **NUMBERS, **kw}
    desc = a.pop("desc") if "desc" in kw else _desc()
    args = [ctypes.byref(desc) if desc is not None else None] + [a[n] for n in CALLS[fn][1:]]
    return getattr(lib, fn)(*args)


@pytest.mark.parametrize("fn", CALLS)
def test_descriptors_and_null_pointers(lib, fn):
    assert call(lib, fn, desc=None) == pa.PA_ERR_NULL
    assert call(lib, fn, desc=_desc(dtype=7)) == pa.PA_ERR_DTYPE
    assert call(lib, fn, desc=_desc(head_dim=96)) == pa.PA_ERR_UNSUPPORTED
    assert call(lib, fn, desc=_desc(num_q_heads=15)) == pa.PA_ERR_SHAPE
    optional = {"refs", "slots", "workspace", "stream"} if fn not in ("pa_share_pages", "pa_extend_tables") else \
        {"stream"} if fn == "pa_share_pages" else {"refs", "stream"}
    for n in CALLS[fn][1:]:
        if n not in NUMBERS and n not in optional:
            assert call(lib, fn, **{n: None}) == pa.PA_ERR_NULL, n
    if fn == "pa_share_pages":
        assert call(lib, fn, refs=None) == pa.PA_ERR_NULL


@pytest.mark.parametrize("fn", ATTENTION)
def test_attention_bounds(lib, fn):
    windowed = "window" in CALLS[fn]
    if windowed:
        for w, s in ((0, 4), (-1, 4), (64, -1), (-(1 << 31), 0)):
            assert call(lib, fn, window=w, sinks=s) == pa.PA_ERR_SHAPE
    assert call(lib, fn, batch=-1) == pa.PA_ERR_SHAPE
    assert call(lib, fn, max_context_len=129) == pa.PA_ERR_SHAPE      # beyond the tables
    assert call(lib, fn, max_context_len=0) == pa.PA_ERR_SHAPE
    assert call(lib, fn, max_pages=0) == pa.PA_ERR_SHAPE
    assert call(lib, fn, scale=float("inf")) == pa.PA_ERR_SHAPE
    for n in ("q", "k_cache", "v_cache", "out"):
        assert call(lib, fn, **{n: FAKE + 8}) == pa.PA_ERR_ALIGN
    assert call(lib, fn, workspace=FAKE + 16) == pa.PA_ERR_ALIGN
    if fn != "pa_prefill_varlen_window":
        assert call(lib, fn, workspace=None) == pa.PA_ERR_WORKSPACE
        assert call(lib, fn, max_ctas=-1) == pa.PA_ERR_SHAPE
        assert call(lib, fn, batch=0) == pa.PA_OK
        assert call(lib, fn, batch=0, q=None, out=None, workspace=None) == pa.PA_OK


def test_windowed_step_rows(lib):
    fn = "pa_decode_kv_write_window"
    assert call(lib, fn, k_stride=1023) == pa.PA_ERR_SHAPE
    assert call(lib, fn, v_stride=1028) == pa.PA_ERR_ALIGN
    assert call(lib, fn, k=FAKE + 8) == pa.PA_ERR_ALIGN
    assert call(lib, fn, desc=_desc(num_pages=1 << 27)) == pa.PA_ERR_UNSUPPORTED


def test_windowed_prefill(lib):
    fn = "pa_prefill_varlen_window"
    assert call(lib, fn, num_tokens=0) == pa.PA_OK
    assert call(lib, fn, num_tokens=0, window=0) == pa.PA_ERR_SHAPE
    assert call(lib, fn, batch=0) == pa.PA_ERR_SHAPE                  # tokens without requests
    assert call(lib, fn, max_seqlen_q=129) == pa.PA_ERR_SHAPE
    assert call(lib, fn, scale=-0.1) == pa.PA_ERR_SHAPE
    assert call(lib, fn, scale=0.0) == pa.PA_ERR_SHAPE


def test_shared_prefix(lib):
    fn = "pa_decode_shared_prefix"
    assert call(lib, fn, groups=-1) == pa.PA_ERR_SHAPE
    assert call(lib, fn, max_prefix=-1) == pa.PA_ERR_SHAPE
    assert call(lib, fn, max_prefix=129) == pa.PA_ERR_SHAPE           # longer than the contexts
    assert call(lib, fn, scale=-0.1) == pa.PA_ERR_SHAPE
    assert call(lib, fn, groups=0, cu_groups=None, prefix_lens=None, workspace=None) == pa.PA_ERR_WORKSPACE


def test_workspace_sizes_of_bad_arguments(lib):
    d = ctypes.byref(_desc())
    for a in ((0, 4, 2, 128, 0), (64, -1, 2, 128, 0), (64, 4, 0, 128, 0), (64, 4, 2, 0, 0), (64, 4, 2, 128, -1)):
        assert lib.pa_decode_window_workspace_size(d, *a) == 0
    for a in ((-1, 2, 100, 128, 0), (1, 0, 100, 128, 0), (1, 2, -1, 128, 0), (1, 2, 100, 0, 0), (1, 2, 100, 128, -1)):
        assert lib.pa_decode_shared_prefix_workspace_size(d, *a) == 0
    assert lib.pa_decode_window_workspace_size(None, 64, 4, 2, 128, 0) == 0
    assert lib.pa_decode_shared_prefix_workspace_size(None, 1, 2, 100, 128, 0) == 0


def test_tables(lib):
    for fn in ("pa_extend_tables", "pa_share_pages", "pa_release_pages", "pa_release_window_pages"):
        assert call(lib, fn, batch=-1) == pa.PA_ERR_SHAPE
        assert call(lib, fn, max_pages=0) == pa.PA_ERR_SHAPE
        assert call(lib, fn, desc=_desc(num_pages=1 << 31)) == pa.PA_ERR_UNSUPPORTED
    assert call(lib, "pa_extend_tables", max_tokens=-1) == pa.PA_ERR_SHAPE
    assert call(lib, "pa_extend_tables", max_tokens=1 << 31) == pa.PA_ERR_SHAPE
    assert call(lib, "pa_share_pages", batch=0) == pa.PA_OK
    for fn in ("pa_release_pages", "pa_release_window_pages"):
        assert call(lib, fn, batch=32769) == pa.PA_ERR_UNSUPPORTED
        assert call(lib, fn, batch=1024, max_pages=1 << 20) == pa.PA_ERR_UNSUPPORTED
    for w, s in ((0, 4), (64, -1)):
        assert call(lib, "pa_release_window_pages", window=w, sinks=s) == pa.PA_ERR_SHAPE


# ---------------------------------------------------------------------------
# run_step with a window, and with groups
# ---------------------------------------------------------------------------
@pytest.fixture
def enqueued(monkeypatch):
    """The calls of the library that a step makes, recorded in place of made."""
    pytest.importorskip("torch")
    from paged_kv_gqa_08_gb300 import step
    calls = []
    for name in [n for n in vars(step) if n.startswith("pa_")]:
        if name.endswith("workspace_size"):
            monkeypatch.setattr(step, name, lambda *a: 4096)
        else:
            monkeypatch.setattr(step, name, lambda *a, name=name, **k: calls.append(name))
    return calls


def _step_args(kind="decode", **kw):
    import torch
    from paged_kv_gqa_08_gb300.step import alloc_step_buffers

    desc = _desc(num_pages=8)
    bufs = alloc_step_buffers(desc, kind, 6, 2, 64, "cpu", norm=True, max_seqlen_q=8, window=16)
    base = torch.zeros(8192, dtype=torch.uint8)
    at = -base.data_ptr() % 256
    bufs.workspace = base[at: at + 4096]
    n = 6 if kind == "prefill" else 2
    cache = torch.zeros(8, 16, 8, 128, dtype=torch.bfloat16)
    rows = torch.zeros(n, 8, 128, dtype=torch.bfloat16)
    a = dict(desc=desc, kind=kind, bufs=bufs, q=torch.zeros(n, 16, 128, dtype=torch.bfloat16), k=rows, v=rows,
             cu_seqlens_q=torch.tensor([0, n // 2, n], dtype=torch.int32),
             context_lens=torch.tensor([20, 30], dtype=torch.int32),
             block_tables=torch.zeros(2, 4, dtype=torch.int32), k_cache=cache, v_cache=cache, scale=0.1,
             max_pages_per_seq=4, max_context_len=64, max_seqlen_q=8)
    a.update(kw)
    return a


def _groups():
    import torch
    return dict(cu_groups=torch.tensor([0, 2], dtype=torch.int32), prefix_lens=torch.tensor([16], dtype=torch.int32),
                max_prefix_len=16)


def _spoil(name):
    import torch

    def odd(t):
        return torch.zeros(t.numel() + 8, dtype=t.dtype)[1: 1 + t.numel()].view(t.shape)

    return {
        "one norm weight": lambda a: a.update(q_norm_w=torch.ones(128, dtype=torch.bfloat16)),
        "unpacked queries": lambda a: a.update(q=torch.zeros(a["q"].shape[0], 32, 128, dtype=torch.bfloat16)[:, :16]),
        "past the tables": lambda a: a.update(max_context_len=65),
        "no length": lambda a: a.update(max_context_len=0, max_prefix_len=0),
        "scale": lambda a: a.update(scale=float("nan")),
        "queries' address": lambda a: a.update(q=odd(a["q"])),
        "output's address": lambda a: setattr(a["bufs"], "out", odd(a["bufs"].out)),
        "workspace": lambda a: setattr(a["bufs"], "workspace", a["bufs"].workspace[:4095]),
        "workspace's address": lambda a: setattr(a["bufs"], "workspace", odd(torch.zeros(5000, dtype=torch.uint8))),
    }[name]


STATUS = {"one norm weight": pa.PA_ERR_NULL, "queries' address": pa.PA_ERR_ALIGN, "output's address": pa.PA_ERR_ALIGN,
          "workspace": pa.PA_ERR_WORKSPACE, "workspace's address": pa.PA_ERR_ALIGN}


@pytest.mark.parametrize("name", ["one norm weight", "unpacked queries", "past the tables", "no length", "scale",
                                  "queries' address", "output's address", "workspace", "workspace's address"])
@pytest.mark.parametrize("how", ["window decode", "window prefill", "groups"])
def test_a_step_is_refused_before_anything_is_enqueued(enqueued, how, name):
    from paged_kv_gqa_08_gb300.step import run_step

    a = _step_args("prefill" if how.endswith("prefill") else "decode")
    a.update(_groups() if how == "groups" else dict(window=16, num_sinks=4))
    _spoil(name)(a)
    with pytest.raises(pa.PagedAttnError) as e:
        run_step(**a)
    assert e.value.status == STATUS.get(name, pa.PA_ERR_SHAPE) and not enqueued


@pytest.mark.parametrize("kind,kw,status", [
    ("decode", dict(window=-1), pa.PA_ERR_SHAPE), ("decode", dict(window=4, num_sinks=-1), pa.PA_ERR_SHAPE),
    ("prefill", dict(window=4, scale=0.0), pa.PA_ERR_SHAPE), ("prefill", dict(window=4, max_seqlen_q=65), pa.PA_ERR_SHAPE),
    ("decode", dict(window=4, groups=True), pa.PA_ERR_UNSUPPORTED), ("prefill", dict(groups=True), pa.PA_ERR_UNSUPPORTED),
    ("decode", dict(window=4, q4=True), pa.PA_ERR_UNSUPPORTED), ("decode", dict(groups=True, q4=True), pa.PA_ERR_UNSUPPORTED),
    ("decode", dict(groups=True, prefix_lens=None), pa.PA_ERR_NULL),
    ("decode", dict(groups=True, max_prefix_len=65), pa.PA_ERR_SHAPE),
    ("decode", dict(groups=True, scale=-0.1), pa.PA_ERR_SHAPE)])
def test_windows_and_groups_that_a_step_does_not_take(enqueued, kind, kw, status):
    from paged_kv_gqa_08_gb300.step import run_step

    kw = dict(kw)
    a = _step_args(kind)
    if kw.pop("groups", False):
        a.update(_groups())
    if kw.pop("q4", False):
        a["bufs"].group_size = 32
    a.update(kw)
    with pytest.raises(pa.PagedAttnError) as e:
        run_step(**a)
    assert e.value.status == status and not enqueued


def test_steps_that_are_not_refused(enqueued):
    import torch
    from paged_kv_gqa_08_gb300.step import run_step

    w = torch.ones(128, dtype=torch.bfloat16)
    run_step(**_step_args(window=16))
    assert enqueued == ["pa_slot_mapping", "pa_kv_write", "pa_decode_window"]
    enqueued.clear()
    run_step(**_step_args("prefill", window=16, num_sinks=4, q_norm_w=w, k_norm_w=w))
    assert enqueued == ["pa_prefill_qk_norm_rope_kv_write", "pa_prefill_varlen_window"]
    enqueued.clear()
    run_step(**_step_args(**_groups(), q_norm_w=w, k_norm_w=w))
    assert enqueued == ["pa_prefill_qk_norm_rope_kv_write", "pa_decode_shared_prefix"]
    enqueued.clear()
    a = _step_args("prefill", window=16)
    a["bufs"].workspace = None
    run_step(**a)
    assert enqueued[-1] == "pa_prefill_varlen_window"
    run_step(**_step_args(num_sinks=4))       # no window: a step over everything
    assert enqueued[-1] == "pa_decode"
