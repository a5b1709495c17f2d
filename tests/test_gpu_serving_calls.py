"""What the C++ marshalling leaves to Python: tensors of a wrong type or shape
in any place of any call.  The tensors of wrong types have room for every type,
so that even a call that were made would stay inside them."""
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U

pytestmark = pytest.mark.gpu

B, HQ, H, D, PAGE, PAGES, COLS = 3, 4, 2, 64, 16, 6, 2


def roomy(shape, dtype):
    """Zeros of `dtype` at the start of storage that would hold 64-bit elements."""
    n = torch.Size(shape).numel()
    raw = torch.zeros(8 * n + 256, dtype=torch.uint8, device="cuda")
    return raw[:n * torch.empty((), dtype=dtype).element_size()].view(dtype).view(shape)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def given(cache):
    f8 = cache is torch.float8_e4m3fn
    c = dict(k_cache=roomy((PAGES, H, PAGE, D), cache), v_cache=roomy((PAGES, H, PAGE, D), cache),
             page_table=torch.arange(B * COLS, dtype=torch.int32, device="cuda").view(B, COLS),
             k_scale=roomy((PAGES, H, PAGE), torch.float32) if f8 else None,
             v_scale=roomy((PAGES, H, PAGE), torch.float32) if f8 else None, layout="seq")
    row = torch.bfloat16
    return {
        "cache_write": dict(k=roomy((B, H, D), row), v=roomy((B, H, D), row), **{x: c[x] for x in ("k_cache", "v_cache", "page_table")},
                            seq_lens=i32(1, 2, 3), cu_new=i32(0, 1, 2, 3), k_scale=c["k_scale"], v_scale=c["v_scale"],
                            layout="seq"),
        "cache_read": dict(k_cache=c["k_cache"], v_cache=c["v_cache"], page_table=c["page_table"], cu_seqlens=i32(0, 1, 2, 3),
                           T=B, first=i32(0, 1, 2), k_scale=c["k_scale"], v_scale=c["v_scale"], dtype=None, layout="seq",
                           out=(roomy((B, H, D), row), roomy((B, H, D), row))),
        "attn_decode": dict(q=roomy((B, HQ, D), row), k_cache=c["k_cache"], v_cache=c["v_cache"], page_table=c["page_table"],
                            seq_lens=i32(1, 2, 3), k_scale=c["k_scale"], v_scale=c["v_scale"], scale=None, layout="seq",
                            workspace=None, out=roomy((B, HQ, D), row), lse=roomy((B, HQ), torch.float32)),
    }


TYPES = (torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float16, torch.int32, torch.int64, torch.uint8)


def wrong(name, t):
    """Tensors like t that are not what the call wants there."""
    for dt in TYPES:
        if dt is not t.dtype:
            yield f"{name} of {dt}", roomy(t.shape, dt)
    if t.dim() > 1:                                  # lengths and offsets count by their elements, in any shape
        yield f"{name} with one dimension more", t[None]
    if name != "page_table":                         # a table may have any number of columns
        yield f"{name} cut", t[..., :-1].contiguous()
    if t.shape[0] > 1:
        yield f"{name} cut in front", t[:-1]
    yield f"{name} on the host", t.cpu()
    if t.dim() > 1:
        yield f"{name} not contiguous", torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device="cuda")[..., ::2]
    yield f"{name} of no tensor", "x"


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("call", ["cache_write", "cache_read", "attn_decode"])
def test_wrong_tensors_are_left_to_python(call, cache):
    U.lib()
    assert U._fast is not None
    fn = getattr(U._fast, call)
    args = given(cache)[call]
    got = fn(*args.values())
    assert got is not None and (type(got) is not int or got == 0)      # the call itself is a plain one
    launches = U.launch_count()
    tried = 0
    for name, t in list(args.items()):
        if not isinstance(t, torch.Tensor):
            continue
        # rows of another type are a plain call, which the library refuses
        for what, bad in wrong(name, t):
            r = fn(*{**args, name: bad}.values())
            assert r is None or (type(r) is int and r != 0), (call, what)
            tried += 1
    if call == "cache_read":
        k, v = args["out"]
        for bad in ((k, v.float()), (k.float(), v), (k[:2], v[:2]), (k, v[:2]), (k, v, v), [k, v], (k, v.cpu()), (k,)):
            assert fn(*{**args, "out": bad}.values()) is None
    torch.cuda.synchronize()
    assert U.launch_count() == launches and tried >= 40
    U.check()


@pytest.mark.parametrize("kt,vt", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float8_e4m3fn),
                                   (torch.bfloat16, torch.float32), (torch.float8_e4m3fn, torch.bfloat16)])
def test_caches_of_two_types_are_refused(kt, vt):
    args = given(torch.bfloat16)
    kc, vc = roomy((PAGES, H, PAGE, D), kt), roomy((PAGES, H, PAGE, D), vt)
    launches = U.launch_count()
    for call, a in args.items():
        a = {**a, "k_cache": kc, "v_cache": vc}
        assert getattr(U._fast, call)(*a.values()) is None
        with pytest.raises(ValueError, match="one shape and dtype"):
            getattr(U, call)(**a)
    assert U.launch_count() == launches
