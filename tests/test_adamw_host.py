"""CPU-only checks of AdamW's entry points and of its plans: every refusal happens
on the host, before anything touches a device."""
import ctypes

import pytest
import torch

import orthonormal_optimizer_step_gb300 as od
from orthonormal_optimizer_step_gb300 import adamw
from orthonormal_optimizer_step_gb300 import build as odbuild

BAD, OK, UNSUPPORTED, NOSPACE = od.DION_ERR_INVALID_ARG, od.DION_OK, od.DION_ERR_UNSUPPORTED, od.DION_ERR_WORKSPACE
P = 1 << 20                                        # an address that is never read: validation fails first


@pytest.fixture(scope="module")
def lib():
    odbuild.build()
    return od.lib()


def tensor(**kw):
    a = dict(n=100, p=P, g=P, m=P, v=P, m_scale=None, v_scale=None, copy=None, p_type=0, g_type=1, lr_factor=1.0, decay_factor=1.0)
    assert set(kw) <= set(a)
    a.update(kw)
    return adamw._Tensor(*a.values())


def table(*tensors):
    return (adamw._Tensor * len(tensors))(*tensors)


def test_structure_is_as_long_as_the_header_says():
    assert ctypes.sizeof(adamw._Tensor) == 8 * 8 + 4 * 4


def step(lib, t, count=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1, step=1, seed=0, scale=None):
    return lib.dion_adamw_step(count, t, lr, b1, b2, eps, wd, step, seed, scale, None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(p=P + 2), dict(g=P + 1), dict(m=P + 2),
    dict(v=P + 2), dict(p_type=2), dict(g_type=-1), dict(m_scale=P), dict(v_scale=P), dict(m_scale=P + 2, v_scale=P),
    dict(copy=P, p_type=1), dict(copy=P + 1), dict(lr_factor=float("nan")), dict(decay_factor=float("inf")),
])
def test_step_refuses_tensors(lib, kw):
    bad = table(tensor(n=0), tensor(**kw))
    hyper = (ctypes.c_double * 5)()
    assert step(lib, bad, 2) == BAD
    assert lib.dion_adamw_step_dev(2, bad, ctypes.addressof(hyper), P, 0, None, P, 256, None) == BAD


def test_step_refuses_numbers(lib):
    t = table(tensor(n=0))
    assert step(lib, t) == OK
    for kw in (dict(lr=float("nan")), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=float("nan")), dict(eps=-1.0),
               dict(eps=float("inf")), dict(wd=float("inf")), dict(step=0), dict(scale=P + 2), dict(count=-1)):
        assert step(lib, t, **kw) == BAD
    assert step(lib, None) == BAD and step(lib, None, 0) == OK
    assert step(lib, table(tensor(n=(1 << 38) + 1))) == UNSUPPORTED


def test_step_on_the_device_refuses(lib):
    t = table(tensor(n=0))
    for args, code in (((None, P, 0, None, P, 256), BAD), ((P + 4, P, 0, None, P, 256), BAD), ((P, None, 0, None, P, 256), BAD),
                       ((P, P + 4, 0, None, P, 256), BAD), ((P, P, 0, P + 1, P, 256), BAD), ((P, P, 0, None, None, 256), NOSPACE),
                       ((P, P, 0, None, P + 8, 256), NOSPACE), ((P, P, 0, None, P, 255), NOSPACE)):
        assert lib.dion_adamw_step_dev(1, t, *args, None) == code


def test_norm_refuses(lib):
    t = table(tensor())
    size = ctypes.c_size_t()
    assert lib.dion_grad_norm_workspace_size(-1, ctypes.byref(size)) == BAD
    assert lib.dion_grad_norm_workspace_size(1, None) == BAD
    for bad in (dict(n=-1), dict(g=None), dict(g=P + 1), dict(g_type=3)):
        assert lib.dion_grad_norm(1, table(tensor(**bad)), 1.0, P, P, 1 << 20, None) == BAD
    for args, code in (((0.0, P, P, 1 << 20), BAD), ((float("nan"), P, P, 1 << 20), BAD), ((1.0, None, P, 1 << 20), BAD),
                       ((1.0, P + 2, P, 1 << 20), BAD)):
        assert lib.dion_grad_norm(1, t, *args, None) == code


# ------------------------------------------------------------------ plans
@pytest.fixture
def on_cpu(monkeypatch):
    """Plans of CPU tensors: what they check of a device's tensors is the same."""
    monkeypatch.setattr(adamw, "_cuda", lambda t, what: 0)
    monkeypatch.setattr(adamw, "_same_device", lambda dev, **tensors: None)


def parts(n=300, p=torch.float32, g=torch.float32, bits=32):
    params, grads = [torch.zeros(n, dtype=p)], [torch.zeros(n, dtype=g)]
    return params, grads, *od.dion_adamw_state(params, bits=bits)


def test_plan_holds_what_the_library_reads(on_cpu):
    p, g, m, v = parts(bits=8, p=torch.bfloat16)
    plan = od.dion_adamw_plan(p, g, m, v, lr_factors=[0.5], decay_factors=[0.0])
    e = plan.table[0]
    assert (e.n, e.p, e.g, e.m, e.m_scale) == (300, p[0].data_ptr(), g[0].data_ptr(), m[0].data.data_ptr(), m[0].scale.data_ptr())
    assert (e.p_type, e.g_type, e.lr_factor, e.decay_factor) == (1, 0, 0.5, 0.0)
    assert m[0].scale.numel() == 2 and not m[0].data.view(torch.uint8).any()
    new = [torch.ones(300, dtype=torch.bfloat16)]
    plan.set_gradients(new)
    assert (e.g, e.g_type) == (new[0].data_ptr(), 1)


def test_plan_refuses(on_cpu):
    p, g, m, v = parts()
    plan = od.dion_adamw_plan
    with pytest.raises(ValueError, match="1 gradients for 2"):
        plan(p * 2, g, m, v)
    with pytest.raises(ValueError, match="shape"):
        plan(p, [torch.zeros(3, 100)], m, v)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        plan([p[0].half()], g, m, v)
    with pytest.raises(TypeError, match="gradient 0 must be float32 or bfloat16"):
        plan(p, [g[0].half()], m, v)
    with pytest.raises(TypeError, match="first moment 0"):
        plan(p, g, [m[0].double()], v)
    with pytest.raises(ValueError, match="second moment 0 has 299"):
        plan(p, g, m, [v[0][1:]])
    with pytest.raises(ValueError, match="contiguous"):
        plan([torch.zeros(600)[::2]], g, m, v)
    m8, v8 = od.dion_adamw_state(p, bits=8)
    with pytest.raises(TypeError, match="both"):
        plan(p, g, m8, v)
    with pytest.raises(ValueError, match="scale has 1"):
        plan(p, g, [od.State8(m8[0].data, m8[0].scale[1:])], v8)
    with pytest.raises(TypeError, match="scales must be float32"):
        plan(p, g, [od.State8(m8[0].data, m8[0].scale.double())], v8)
    with pytest.raises(TypeError, match="copy 0"):
        plan(p, g, m, v, copies=[torch.zeros(300)])
    with pytest.raises(ValueError, match="finite"):
        plan(p, g, m, v, lr_factors=[float("inf")])
    with pytest.raises(ValueError, match="bits"):
        od.dion_adamw_state(p, bits=16)


def test_plan_refuses_shared_memory(on_cpu):
    p, g, m, v = parts()
    plan = od.dion_adamw_plan
    with pytest.raises(ValueError, match="share memory"):
        plan(p * 2, g * 2, m * 2, v * 2)                                 # the same tensor twice
    with pytest.raises(ValueError, match="share memory"):
        plan(p, g, m, m)
    with pytest.raises(ValueError, match="gradient shares"):
        plan(p, p, m, v)
    both = torch.zeros(599)
    with pytest.raises(ValueError, match="share memory"):
        plan([both[:300]], g, [both[299:]], v)
    kept = plan(p, g, m, v)
    at = kept.table[0].g
    with pytest.raises(ValueError, match="gradient shares"):
        kept.set_gradients(v)
    assert kept.table[0].g == at and kept.tensors[0] is not v            # as it was
    plan(p + [torch.zeros(4)], g + [g[0][:4]], m + [torch.zeros(4)], v + [torch.zeros(4)])   # gradients may be shared


def test_plan_keeps_the_memory_that_it_writes(on_cpu):
    """A tensor that is given other memory lets go of what the plan's table points to; the plan does not."""
    p, g, m, v = parts(bits=8)
    plan = od.dion_adamw_plan(p, g, m, v, copies=[torch.zeros(300, dtype=torch.bfloat16)])
    later = [torch.zeros(300)]
    for t in (p[0], g[0], m[0].data, m[0].scale, v[0].data, v[0].scale):
        t.data = torch.ones_like(t)
    e, (kept_g, kept_p, kept_m, kept_v, kept_c) = plan.table[0], [x[0] for x in plan.tensors]
    assert (e.p, e.g, e.copy) == (kept_p.data_ptr(), kept_g.data_ptr(), kept_c.data_ptr())
    assert (e.m, e.m_scale, e.v, e.v_scale) == (kept_m.data.data_ptr(), kept_m.scale.data_ptr(), kept_v.data.data_ptr(), kept_v.scale.data_ptr())
    plan.set_gradients(later)
    later[0].data = torch.ones(300)
    assert e.g == plan.tensors[0][0].data_ptr() != later[0].data_ptr()
    listed = od.dion_grad_list(later)
    later[0].data = torch.zeros(300)
    assert listed.table[0].g == listed.tensors[0][0].data_ptr() != later[0].data_ptr()


def test_gradients_on_the_cpu_are_refused():
    with pytest.raises(ValueError, match="CUDA"):
        od.dion_grad_list([torch.zeros(4)])
