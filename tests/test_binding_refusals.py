"""Refusals of the native entry points: each names the argument, before anything is launched."""
import pytest
import torch

from quantized_routed_expert_02_gb300 import moeq4k as m

F32, F16, BF16, I32, I8 = torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.int8


def norm_args():
    return dict(x=torch.zeros(2, 256), residual=torch.zeros(2, 256), gamma=torch.zeros(256), eps=1e-6,
                sum_out=torch.zeros(2, 256), y=torch.zeros(2, 256, dtype=BF16),
                q8k=(torch.zeros(2, 256, dtype=I8), torch.zeros(2, 1), torch.zeros(2, 8, dtype=I32)), stream=0)


def cache_args(dtype):
    return dict(k_pages=torch.zeros(4, 2, 16, 64, dtype=dtype), v_pages=torch.zeros(4, 2, 16, 64, dtype=dtype),
                page_table=torch.zeros(1, 2, dtype=I32), q_offs=torch.tensor([0, 3], dtype=I32),
                kv_lens=torch.tensor([5], dtype=I32), ws=torch.zeros(1 << 20, dtype=torch.uint8), stream=0)


def rope_args():
    return dict(cache_args(F16), qkv=torch.zeros(3, 8 * 64, dtype=F16), pos=torch.zeros(1, 3, dtype=I32),
                inv_freq=torch.zeros(16, dtype=torch.float64), q_out=torch.zeros(3, 4, 64, dtype=F16),
                axis=torch.zeros(16, dtype=I32), q_norm_w=torch.zeros(64), k_norm_w=torch.zeros(64))


def attn_args():
    return dict(cache_args(BF16), q=torch.zeros(3, 4, 64, dtype=BF16), max_new=3, scale=0.125,
                out=torch.zeros(3, 4, 64, dtype=BF16), lse=torch.zeros(3, 4))


CALLS = {"moe_add_rmsnorm": norm_args, "moe_rope_append": rope_args, "moe_attention_paged": attn_args}
BAD = [
    ("moe_add_rmsnorm", "x", torch.zeros(256), ValueError),
    ("moe_add_rmsnorm", "x", torch.zeros(2, 256, dtype=torch.float64), TypeError),
    ("moe_add_rmsnorm", "residual", torch.zeros(2, 256, dtype=BF16), TypeError),
    ("moe_add_rmsnorm", "residual", torch.zeros(3, 256), ValueError),
    ("moe_add_rmsnorm", "gamma", torch.zeros(512)[::2], ValueError),
    ("moe_add_rmsnorm", "gamma", None, TypeError),
    ("moe_add_rmsnorm", "y", torch.zeros(2, 512)[:, ::2], ValueError),
    ("moe_add_rmsnorm", "q8k", (torch.zeros(2, 256, dtype=I8), torch.zeros(2, 1)), TypeError),
    ("moe_add_rmsnorm", "eps", "small", TypeError),
    ("moe_rope_append", "qkv", torch.zeros(3, 7 * 64, dtype=F16), ValueError),
    ("moe_rope_append", "qkv", torch.zeros(3, 8 * 64, dtype=BF16), TypeError),
    ("moe_rope_append", "pos", torch.zeros(1, 2, dtype=I32), ValueError),
    ("moe_rope_append", "pos", torch.zeros(1, 3, dtype=torch.int64), TypeError),
    ("moe_rope_append", "inv_freq", torch.zeros(16), TypeError),
    ("moe_rope_append", "axis", torch.zeros(15, dtype=I32), ValueError),
    ("moe_rope_append", "q_out", torch.zeros(3, 4, 128, dtype=F16), ValueError),
    ("moe_rope_append", "k_norm_w", torch.zeros(128), ValueError),
    ("moe_rope_append", "k_pages", torch.zeros(4, 2, 64, 16, dtype=F16).transpose(2, 3), ValueError),
    ("moe_rope_append", "v_pages", torch.zeros(3, 2, 16, 64, dtype=F16), ValueError),
    ("moe_attention_paged", "q", torch.zeros(3, 4 * 64, dtype=BF16), ValueError),
    ("moe_attention_paged", "v_pages", torch.zeros(4, 2, 16, 64, dtype=F16), TypeError),
    ("moe_attention_paged", "page_table", torch.zeros(1, 2, dtype=torch.int64), TypeError),
    ("moe_attention_paged", "q_offs", torch.zeros(3, dtype=I32), ValueError),
    ("moe_attention_paged", "kv_lens", torch.zeros(2, dtype=I32), ValueError),
    ("moe_attention_paged", "out", torch.zeros(3, 4, 64, dtype=F16), TypeError),
    ("moe_attention_paged", "lse", torch.zeros(4, 3), ValueError),
    ("moe_attention_paged", "ws", 5, TypeError),
]


@pytest.mark.parametrize("call,name,value,error", BAD)
def test_bad_argument(call, name, value, error):
    with pytest.raises(error) as e:
        getattr(m, call)(**dict(CALLS[call](), **{name: value}))
    assert name in str(e.value) or name in ("eps",)


@pytest.mark.parametrize("call", CALLS)
def test_argument_lists(call):
    args = CALLS[call]()
    with pytest.raises(TypeError, match="unexpected keyword"):
        getattr(m, call)(**args, other=1)
    with pytest.raises(TypeError, match="missing argument"):
        getattr(m, call)(next(iter(args.values())))
    with pytest.raises(TypeError, match="takes"):
        getattr(m, call)(*range(40))
    with pytest.raises(TypeError, match="multiple values"):
        getattr(m, call)(*range(5), **args)


@pytest.mark.parametrize("call,change,status", [
    ("moe_add_rmsnorm", dict(eps=-1.0), "MOE_ERR_INVALID_SHAPE"),
    ("moe_add_rmsnorm", dict(sum_out=None, y=None, q8k=None), "MOE_ERR_NULL"),
    ("moe_rope_append", dict(inv_freq=torch.zeros(15, dtype=torch.float64), axis=None), "MOE_ERR_INVALID_SHAPE"),
    ("moe_attention_paged", dict(max_new=0), "MOE_ERR_INVALID_SHAPE"),
    ("moe_attention_paged", dict(scale=float("nan")), "MOE_ERR_INVALID_SHAPE"),
    ("moe_attention_paged", dict(ws=torch.zeros(256, dtype=torch.uint8)), "MOE_ERR_WORKSPACE")])
def test_the_library_refuses(call, change, status):
    args = dict(CALLS[call](), **change)
    for name, t in args.items():  # the library asks for aligned pointers, which the host may not give
        if isinstance(t, torch.Tensor) and t.data_ptr() % 256:
            big = torch.zeros(t.nbytes + 256, dtype=torch.uint8)
            at = -big.data_ptr() % 256
            args[name] = big[at:at + t.nbytes].view(t.dtype).view(t.shape).copy_(t)
    with pytest.raises(m.MoeError, match=status):
        getattr(m, call)(**args)


def test_integers_past_32_bits():
    with pytest.raises(OverflowError):
        m.moe_attention_paged(**dict(attn_args(), max_new=1 << 40))


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
def test_a_tensor_left_on_the_host(call):
    """Every tensor in turn: refused before a kernel could see its address."""
    def to(v, dev):
        return tuple(to(t, dev) for t in v) if isinstance(v, tuple) else v.to(dev) if isinstance(v, torch.Tensor) else v

    args = {k: to(v, "cuda") for k, v in CALLS[call]().items()}
    del args["stream"]
    for name, v in CALLS[call]().items():
        if isinstance(v, (torch.Tensor, tuple)):
            with pytest.raises(ValueError, match="on c"):
                getattr(m, call)(**dict(args, **{name: v}))


def on_aligned_storage(args):
    """The same arguments on storage aligned as a device's would be."""
    def align(t):
        big = torch.zeros(t.nbytes + 256, dtype=torch.uint8)
        at = -big.data_ptr() % 256
        return big[at:at + t.nbytes].view(t.dtype).view(t.shape).copy_(t)

    def to(v):
        return tuple(map(to, v)) if isinstance(v, tuple) else align(v) if isinstance(v, torch.Tensor) else v

    args = {k: to(v) for k, v in args.items()}
    if "ws" in args:
        args["ws"] = align(torch.zeros(48 << 20, dtype=torch.uint8))
    return args


@pytest.mark.parametrize("stream", [0, None, 1 << 20])
@pytest.mark.parametrize("call", CALLS)
def test_all_tensors_on_the_host(call, stream):
    """Right in all but their place: refused, whatever the stream, before a kernel could see an address."""
    args = dict(on_aligned_storage(CALLS[call]()), stream=stream)
    with pytest.raises(ValueError, match="cpu, which is not the current CUDA device"):
        getattr(m, call)(**args)


@pytest.mark.parametrize("call", ["moe_rope_append", "moe_attention_paged"])
@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(48 << 20),
                                torch.zeros(2 << 20, dtype=torch.uint8)[::2]], ids=["expanded", "strided"])
def test_a_workspace_that_is_no_run_of_bytes(call, ws):
    with pytest.raises(ValueError, match="ws: not contiguous"):
        getattr(m, call)(**dict(CALLS[call](), ws=ws))


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
def test_a_stream_that_is_none(call):
    """The handle that stands for checking alone is no stream of a caller's."""
    args = {k: v.to("cuda") if isinstance(v, torch.Tensor) else v for k, v in CALLS[call]().items() if k != "q8k"}
    with pytest.raises(ValueError, match="stream"):
        getattr(m, call)(**dict(args, stream=-1))
