"""Refusals of the norm, block-scale and block-attention calls (no GPU): through the C ABI,
and of tensors by the Python calls (types, shapes, layouts; the device is looked at last)."""

import pytest
import torch

from paged_kv_cache_55_gb300 import binding as B
from paged_kv_cache_55_gb300 import build as build_mod

P = 0x10000  # a pointer that no refused call follows
NULL, DIMS, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


NORM = dict(q=P, q_stride=256, key=P, key_stride=128, qw=P, kw=P, eps=1e-6, positions=P, table=P, max_position=100,
            rotary_dim=64, is_neox=1, num_tokens=3, num_heads=4, num_kv_heads=2, head_dim=64, q_out=P + 4096,
            q_out_stride=256, key_out=P + 8192, key_out_stride=128, dtype=0, stream=None)
NORM_REFUSALS = [
    (dict(dtype=2), UNSUPPORTED), (dict(num_tokens=-1), DIMS), (dict(num_heads=0), DIMS), (dict(eps=0.0), DIMS),
    (dict(eps=float("inf")), DIMS), (dict(eps=float("nan")), DIMS), (dict(eps=-1e-6), DIMS),
    (dict(rotary_dim=80), DIMS), (dict(rotary_dim=8), ALIGN), (dict(rotary_dim=0), DIMS),
    (dict(max_position=0), DIMS), (dict(head_dim=68), ALIGN),
    (dict(head_dim=520, q_stride=4096, key_stride=4096, q_out_stride=4096, key_out_stride=4096), UNSUPPORTED),
    (dict(q=None), NULL), (dict(key=None), NULL), (dict(q_out=None), NULL), (dict(key_out=None), NULL),
    (dict(positions=None), NULL), (dict(table=None), NULL), (dict(q_stride=248), DIMS), (dict(key_stride=120), DIMS),
    (dict(q_out_stride=248), DIMS), (dict(key_out_stride=120), DIMS), (dict(q_stride=260), ALIGN),
    (dict(q=P + 8), ALIGN), (dict(qw=P + 8), ALIGN), (dict(kw=P + 2), ALIGN), (dict(table=P + 4), ALIGN),
    (dict(positions=P + 4), ALIGN), (dict(q_out=P, q_out_stride=264), DIMS),
    (dict(key_out=P, key_out_stride=136), DIMS), (dict(num_heads=1 << 29), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", NORM_REFUSALS, ids=lambda v: str(v))
def test_norm_rope_refusals(lib, change, status):
    assert lib.pa_norm_rope(*{**NORM, **change}.values()) == status
    assert lib.pa_launch_count() == 0


def test_norm_rope_of_no_tokens_launches_nothing(lib):
    none = dict(num_tokens=0, q=None, key=None, q_out=None, key_out=None, positions=None, table=None, qw=None, kw=None)
    assert lib.pa_norm_rope(*{**NORM, **none}.values()) == 0


CACHE = dict(q=P, q_stride=256, key=P, value=P, key_stride=128, value_stride=128, qw=None, kw=P, eps=1e-6, kc=P, vc=P,
             slots=P, positions=P, table=P, max_position=100, rotary_dim=64, is_neox=0, num_tokens=3, num_heads=4,
             num_kv_heads=2, head_dim=64, block_size=16, num_blocks=10)


@pytest.mark.parametrize("change,status", [
    (dict(value=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(slots=None), NULL),
    (dict(value_stride=64), DIMS), (dict(block_size=0), DIMS), (dict(num_blocks=-1), DIMS), (dict(kc=P + 4), ALIGN),
    (dict(slots=P + 4), ALIGN), (dict(num_blocks=(1 << 62), block_size=16), UNSUPPORTED), (dict(head_dim=66), ALIGN),
], ids=lambda v: str(v))
def test_norm_rope_cache_refusals(lib, change, status):
    args = {**CACHE, **change}
    assert lib.pa_norm_rope_reshape_and_cache(*args.values(), P, 256, 1, None) == status
    assert lib.pa_norm_rope_reshape_and_cache_fp8(*args.values(), 0.1, 0.1, P, 256, 1, None) == status


def test_norm_rope_cache_scales(lib):
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("inf"), 1.0), (1.0, float("nan"))):
        assert lib.pa_norm_rope_reshape_and_cache_fp8(*CACHE.values(), ks, vs, P, 256, 0, None) == DIMS
    odd = {**CACHE, "head_dim": 72}  # 8-bit rows are whole 16-byte vectors
    assert lib.pa_norm_rope_reshape_and_cache_fp8(*odd.values(), 1.0, 1.0, P, 1024, 0, None) == ALIGN


SCATTER = dict(key=P, value=P, key_stride=128, value_stride=128, kc=P, vc=P, ks=P, vs=P, tables=P, max_blocks=4, lens=P,
               starts=P, num_seqs=2, total=5, max_query=3, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=10,
               dtype=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(num_seqs=-1), DIMS), (dict(total=-1), DIMS), (dict(max_query=-1), DIMS),
    (dict(max_query=0), DIMS), (dict(max_query=6), DIMS), (dict(max_blocks=0), DIMS), (dict(num_blocks=0), DIMS),
    (dict(head_dim=112), UNSUPPORTED), (dict(block_size=64), UNSUPPORTED), (dict(key=None), NULL),
    (dict(value=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(ks=None), NULL),
    (dict(vs=None), NULL), (dict(tables=None), NULL), (dict(lens=None), NULL), (dict(starts=None), NULL),
    (dict(key_stride=120), DIMS), (dict(value_stride=130), ALIGN), (dict(ks=P + 2), ALIGN), (dict(kc=P + 8), ALIGN),
    (dict(tables=P + 2), ALIGN), (dict(num_seqs=1 << 30), UNSUPPORTED), (dict(num_kv_heads=1 << 26), UNSUPPORTED),
    (dict(num_seqs=0), 0), (dict(total=0), 0),
], ids=lambda v: str(v))
def test_block_scatter_refusals(lib, change, status):
    assert lib.pa_reshape_and_cache_fp8_block(*{**SCATTER, **change}.values()) == status
    assert lib.pa_launch_count() == 0


ATTENTION = dict(q=P, q_stride=512, kc=P, vc=P, ks=P, vs=P, tables=P, max_blocks=4, lens=P, starts=P, num_seqs=2,
                 total=2, max_query=1, max_len=60, num_heads=8, num_kv_heads=2, head_dim=64, block_size=16,
                 num_blocks=10, scale=0.125, out=P, workspace=P, workspace_bytes=1 << 30, dtype=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(scale=0.0), DIMS), (dict(scale=-0.1), DIMS), (dict(scale=float("nan")), DIMS),
    (dict(scale=float("inf")), DIMS), (dict(ks=None), NULL), (dict(vs=None), NULL), (dict(ks=P + 2), ALIGN),
    (dict(vs=P + 1), ALIGN), (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=None), WORKSPACE),
    (dict(workspace=P + 128), ALIGN), (dict(head_dim=112), UNSUPPORTED), (dict(num_heads=24), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(q=None), NULL), (dict(out=P + 8), ALIGN), (dict(num_seqs=0), 0),
], ids=lambda v: str(v))
def test_block_attention_refusals(lib, change, status):
    assert lib.pa_attention_varlen_fp8_block(*{**ATTENTION, **change}.values()) == status
    assert lib.pa_launch_count() == 0


def test_copy_block_scales_refusals(lib):
    f = lib.pa_copy_block_scales
    assert f(P, P, P, -1, 2, 10, None) == DIMS
    assert f(P, P, P, 1, 0, 10, None) == DIMS
    assert f(None, P, P, 1, 2, 10, None) == NULL
    assert f(P, P, P + 4, 1, 2, 10, None) == ALIGN
    assert f(None, None, None, 0, 2, 10, None) == 0


# ---- tensors ---------------------------------------------------------------

def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def norm_args(**change):
    a = dict(q=z(3, 4, 64), key=z(3, 2, 64), q_weight=z(64), k_weight=None, eps=1e-6,
             positions=z(3, dtype=torch.int64), cos_sin_cache=z(10, 64, dtype=torch.float32), q_out=z(3, 4, 64),
             key_out=z(3, 2, 64))
    a.update(change)
    return a


def cache_args(cache=torch.bfloat16, **change):
    a = dict(q=z(3, 4, 64), key=z(3, 2, 64), value=z(3, 2, 64), q_weight=None, k_weight=z(64), eps=1e-6,
             key_cache=z(5, 16, 2, 64, dtype=cache), value_cache=z(5, 16, 2, 64, dtype=cache),
             slot_mapping=z(3, dtype=torch.int64), positions=z(3, dtype=torch.int64),
             cos_sin_cache=z(10, 64, dtype=torch.float32), q_out=z(3, 4, 64))
    a.update(change)
    return a


def scatter_args(**change):
    a = dict(key=z(5, 2, 64), value=z(5, 2, 64), key_cache=z(6, 16, 2, 64, dtype=torch.uint8),
             value_cache=z(6, 16, 2, 64, dtype=torch.uint8), k_scales=z(6, 2, dtype=torch.float32),
             v_scales=z(6, 2, dtype=torch.float32), block_tables=z(2, 4, dtype=torch.int32),
             seq_lens=z(2, dtype=torch.int32), query_start_loc=z(3, dtype=torch.int32), max_query_len=3)
    a.update(change)
    return a


def attention_args(**change):
    a = scatter_args()
    del a["key"], a["value"]
    a.update(q=z(5, 8, 64), out=z(5, 8, 64), max_seq_len=60, scale=0.1,
             workspace=z(1024, dtype=torch.uint8))
    a.update(change)
    return a


CALLS = {
    "norm_rope": (B.pa_norm_rope, norm_args),
    "norm_rope_cache": (B.pa_norm_rope_reshape_and_cache, cache_args),
    "norm_rope_cache8": (lambda **a: B.pa_norm_rope_reshape_and_cache_fp8(k_scale=1.0, v_scale=1.0, **a),
                         lambda **c: cache_args(torch.uint8, **c)),
    "scatter": (B.pa_reshape_and_cache_fp8_block, scatter_args),
    "attention": (B.pa_attention_varlen_fp8_block, attention_args),
}
WRONG = {
    "norm_rope": [(dict(q=z(3, 4, 64).float()), TypeError), (dict(q=5), TypeError), (dict(key=None), TypeError),
                  (dict(key=z(3, 2, 64).half()), TypeError), (dict(positions=z(3, dtype=torch.int32)), TypeError),
                  (dict(cos_sin_cache=z(10, 64)), TypeError), (dict(key=z(2, 2, 64)), ValueError),
                  (dict(key=z(3, 2, 32)), ValueError), (dict(q=z(3, 256)), ValueError),
                  (dict(q_weight=z(32)), ValueError), (dict(q_weight=z(64).float()), TypeError),
                  (dict(k_weight=z(128)[::2]), ValueError), (dict(positions=z(4, dtype=torch.int64)), ValueError),
                  (dict(q_out=z(3, 4, 32)), ValueError), (dict(key_out=z(3, 4, 64)), ValueError),
                  (dict(q=z(3, 64, 4).transpose(1, 2)), ValueError), (dict(q_out=z(3, 8, 64)[:, ::2]), ValueError),
                  (dict(cos_sin_cache=z(10, 128, dtype=torch.float32)[:, ::2]), ValueError),
                  (dict(eps="x"), TypeError)],
    "norm_rope_cache": [(dict(value=z(3, 3, 64)), ValueError), (dict(key_cache=z(5, 16, 4, 64)), ValueError),
                        (dict(value_cache=z(5, 8, 2, 64)), ValueError),
                        (dict(key_cache=z(5, 16, 2, 64, dtype=torch.uint8)), TypeError),
                        (dict(slot_mapping=z(2, dtype=torch.int64)), ValueError),
                        (dict(slot_mapping=z(3, dtype=torch.int32)), TypeError),
                        (dict(key_cache=z(10, 16, 2, 64)[::2]), ValueError)],
    "norm_rope_cache8": [(dict(key_cache=z(5, 16, 2, 64)), TypeError)],
    "scatter": [(dict(key=z(5, 3, 64)), ValueError), (dict(value=z(4, 2, 64)), ValueError),
                (dict(k_scales=z(6, 3, dtype=torch.float32)), ValueError),
                (dict(v_scales=z(6, 2)), TypeError), (dict(k_scales=z(6, dtype=torch.float32)), ValueError),
                (dict(v_scales=z(2, 6, dtype=torch.float32).t()), ValueError),
                (dict(block_tables=z(3, 4, dtype=torch.int32)), ValueError),
                (dict(seq_lens=z(2, dtype=torch.int64)), TypeError),
                (dict(query_start_loc=z(2, dtype=torch.int32)), ValueError),
                (dict(block_tables=z(4, 2, dtype=torch.int32).t()), ValueError),
                (dict(key_cache=z(6, 16, 2, 64)), TypeError), (dict(max_query_len="3"), TypeError),
                (dict(max_query_len=1 << 40), ValueError)],
    "attention": [(dict(out=z(5, 8, 32)), ValueError), (dict(q=z(5, 8, 32)), ValueError),
                  (dict(out=z(5, 8, 64).half()), TypeError), (dict(out=z(5, 16, 64)[:, ::2]), ValueError),
                  (dict(workspace=None), TypeError), (dict(workspace=z(2048, dtype=torch.uint8)[::2]), ValueError),
                  (dict(max_seq_len=1 << 40), ValueError), (dict(scale=None), TypeError),
                  (dict(v_scales=z(6, 4, dtype=torch.float32)), ValueError)],
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_off_the_gpu_are_refused(lib, name):
    call, args = CALLS[name]
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        call(**args())


@pytest.mark.parametrize("name,change,error", [(n, c, e) for n in sorted(WRONG) for c, e in WRONG[n]],
                         ids=[f"{n}-{i}-{'-'.join(c)}" for n in sorted(WRONG) for i, (c, e) in enumerate(WRONG[n])])
def test_wrong_tensors_are_refused(lib, name, change, error):
    call, args = CALLS[name]
    with pytest.raises(error) as e:
        call(**args(**change))
    assert "must be a CUDA tensor" not in str(e.value) or any(not isinstance(v, torch.Tensor) for v in change.values())
    assert B.pa_launch_count() == 0
