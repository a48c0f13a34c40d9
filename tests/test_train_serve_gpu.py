"""The operators as a program uses them together: 8-bit layers trained with the Dion
step for their matrices and clipped AdamW for the rest, then served in 4 bits."""
import importlib.util
import os

import pytest
import torch

import adamw_ref as ref
import orthonormal_optimizer_step_gb300 as od
import q4_ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "q8_training.py")
F32, BF16 = torch.float32, torch.bfloat16
EPS32 = 2.0 ** -24
LAYERS, WIDTH, TOKENS, WORDS = 3, 256, 384, 500
LR, BETAS, EPS, DECAY, SEED, MAX_NORM = 1e-2, (0.9, 0.999), 1e-8, 0.1, 7, 0.5


class Model:
    """An embedding (8-bit states, a bfloat16 copy that the forward pass reads) and 8-bit layers (float32 states of
    their norms' weights)."""

    def __init__(self):
        spec = importlib.util.spec_from_file_location("q8_training", PATH)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(3)
        self.stack = mod.Stack(LAYERS, WIDTH, seed=2)
        self.table = torch.randn(WORDS, WIDTH, generator=gen, device="cuda") * 0.5
        self.table16 = self.table.to(BF16)
        self.table_grad = torch.zeros_like(self.table)
        (m8,), (v8,) = od.dion_adamw_state([self.table], bits=8)
        (m32,), (v32,) = od.dion_adamw_state([self.stack.norm])
        self.moments = [m8, m32], [v8, v32]
        self.plan = od.dion_adamw_plan([self.table, self.stack.norm], [self.table_grad, self.stack.norm_grad], *self.moments,
                                       copies=[self.table16, None], decay_factors=[1.0, 0.0])
        self.ids = torch.randint(WORDS, (TOKENS,), generator=gen, device="cuda")
        self.target = torch.randn(TOKENS, WIDTH, generator=gen, device="cuda")
        self.hyper = torch.tensor([LR, *BETAS, EPS, DECAY], dtype=torch.float64, device="cuda")
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def gradients(self):
        out, saved = self.stack.forward(self.table16[self.ids])
        dx = self.stack.backward(((out.float() - self.target) / TOKENS).to(BF16), saved)
        # (as a product, whose order of sums does not change from run to run)
        rows = torch.nn.functional.one_hot(self.ids, WORDS).to(F32)
        self.table_grad.copy_(rows.t() @ dx.float())
        return od.dion_grad_norm(self.plan, max_norm=MAX_NORM)

    def update(self, norm):
        s = self.stack
        od.dion_step_batched(s.X, s.G, s.M, s.Q, mu=0.95, lr=LR, weight_decay=0.0)
        od.dion_adamw_step(self.plan, step=self.step, hyper=self.hyper, grad_scale=norm[1:], seed=SEED)
        s.quantize()

    def tensors(self):
        s = self.stack
        (m8, m32), (v8, v32) = self.moments
        return [s.X, s.M, s.Q, s.norm, self.table, self.table16, m8.data.view(torch.uint8), m8.scale, v8.data.view(torch.uint8),
                v8.scale, m32, v32, self.step]


def moments_of(state, n):
    return ref.values(state, n) if isinstance(state, od.State8) else state.double().flatten()


def test_steps_follow_the_formula():
    model = Model()
    for t in range(1, 5):
        norm = model.gradients()
        grads = [model.table_grad.flatten(), model.stack.norm_grad.flatten()]
        want = torch.cat(grads).double().norm()
        assert abs(float(norm[0]) - float(want)) <= 2.0 ** -20 * float(want)     # float32 squares of 64 at a time, float64 sums
        assert abs(float(norm[1]) - min(1.0, MAX_NORM / (float(want) + 1e-6))) <= 2.0 ** -19
        params = [model.table.flatten().clone(), model.stack.norm.flatten().clone()]
        first = [moments_of(x, p.numel()) for x, p in zip(model.moments[0], params)]
        second = [moments_of(x, p.numel()) for x, p in zip(model.moments[1], params)]
        second[0] = second[0].square()
        model.update(norm)
        for i, p in enumerate((model.table, model.stack.norm)):
            new, m, v, size = ref.step(params[i], grads[i], first[i], second[i], t, lr=LR, betas=BETAS, eps=EPS,
                                       weight_decay=(DECAY, 0.0)[i], scale=float(norm[1]))
            # the update's constants, its moments, the root, the quotient and products: 20 half steps; p's own three, and two of its decay
            assert torch.all((p.flatten().double() - new).abs() <= 20 * EPS32 * size + 3 * EPS32 * new.abs() + 2 * EPS32 * params[i].double().abs())
            if i == 0:
                terms = 0.9 * first[0].abs() + 0.1 * (grads[0].double() * float(norm[1])).abs()
                ref.check8(model.moments[0][0], m, terms=terms)
                ref.check8(model.moments[1][0], v.sqrt(), ref.dither(p.numel(), SEED, t, 0))
        assert torch.equal(model.table16, model.table.to(BF16)) and int(model.step) == t


def test_a_captured_training_step_has_the_same_bits():
    """Forward, backward, norm, both optimizers and the weights' quantization in one CUDA graph, replayed."""
    eager, model = Model(), Model()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                          # (the library's own state is set up)
        model.update(model.gradients())
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            model.update(model.gradients())
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
    for _ in range(4):
        eager.update(eager.gradients())
    assert int(model.step) == 4
    for a, b in zip(model.tensors(), eager.tensors()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("group", [32, 128])
def test_serving_the_trained_weights(tokens, group):
    model = Model()
    model.update(model.gradients())
    s = model.stack
    w4 = [od.dion_q4_quantize(s.X[l], group=group) for l in range(LAYERS)]
    delta, r = model.table16[model.ids[:tokens]], None
    for l in range(LAYERS):
        q, scale = q4_ref.groups(s.X[l], group)
        assert torch.equal(w4[l].scale.cpu(), scale) and torch.equal(w4[l].data.cpu(), q4_ref.pack(q))
        x8, r, _ = od.dion_rms_norm_q8(delta, s.norm[l], residual=r)
        delta = od.dion_q4_matmul(x8, w4[l])
        xv = x8.data.double() * torch.exp2(x8.scale.view(torch.uint8).double() - 127).repeat_interleave(128, 1)[:, :WIDTH]
        wv = (q.double() * scale.double().repeat_interleave(group, 1)).cuda()
        want, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
        # products are exact; a sum is at most 16 of the tensor cores (truncated, 2^-23), its groups, chunks and shares; one rounding to bfloat16
        chain = WIDTH / 16 + WIDTH / group + WIDTH / 128 + 16
        assert torch.all((delta.double() - want).abs() <= chain * 2.0 ** -23 * size + 2.0 ** -8 * want.abs())
        # the same where many rows would be multiplied: the values back, in 8 bits, through the other product
        assert torch.equal(od.dion_q4_dequantize(w4[l], out_dtype=F32).double(), wv.float().double())
