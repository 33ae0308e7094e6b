"""A learned stand-in for a block Toeplitz operator that answers one time step
at a time.

F applies to whole series: v = F m needs all of m. A recurrent layer that has
learned F's impulse responses gives each v_t as m_t arrives. This example
draws an operator of decaying modes, F_k = C diag(a^k) B, takes its training
pairs from ``Plan.apply`` on random series, fits a ``layers.RecurrentLayer``
(or, with ``--layer delta``, a ``layers.DeltaLayer``) to them, and then streams
a fresh series through the layer step by step.

    python -m fft_block_toeplitz_amd.surrogate [--layer delta] [--iterations 400] [--steps 200]
"""

from __future__ import annotations

import argparse


def modes_operator(Nm: int, Nd: int, Nt: int, modes: int, generator, device="cuda"):
    """F [Nt][Nd][Nm] float64 with F_k = C diag(a^k) B, memories of 1 to ~50 steps."""
    import torch

    def normal(*shape):
        return torch.randn(shape, generator=generator, device=device, dtype=torch.float64)

    a = torch.linspace(0.2, 0.98, modes, device=device, dtype=torch.float64)
    B, C = normal(modes, Nm) * (1.0 - a * a).sqrt()[:, None] / Nm ** 0.5, normal(Nd, modes) / modes ** 0.5
    k = torch.arange(Nt, device=device, dtype=torch.float64)
    # (k, r) rows of C a^k times B: one product of contiguous matrices
    left = (C[None] * (a[None, :] ** k[:, None])[:, None, :]).reshape(Nt * Nd, modes).contiguous()
    return (left @ B.contiguous()).reshape(Nt, Nd, Nm).contiguous()


def run(iterations: int = 400, Nm: int = 24, Nd: int = 6, Nt: int = 200, batch: int = 16, channels: int = 128,
        seed: int = 0, report=print, layer: str = "recurrent") -> dict:
    """Fits the layer and streams with it; returns the errors, relative L2.
    ``channels``: those of a recurrent layer's state, or the values of all heads
    of a delta layer, 16 a head."""
    import torch

    import fft_block_toeplitz_amd as fm
    from fft_block_toeplitz_amd.layers import DeltaLayer, RecurrentLayer

    if layer not in ("recurrent", "delta"):
        raise ValueError(f"layer must be 'recurrent' or 'delta', got {layer!r}")

    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    torch.manual_seed(seed)
    plan = fm.Plan(modes_operator(Nm, Nd, Nt, 12, gen), fm.FFTMV_ALL_FP64)

    def series(n):
        m = torch.randn((n, Nt, Nm), generator=gen, device="cuda", dtype=torch.float64)
        v = torch.stack([plan.apply(m[i]) for i in range(n)])
        return m.float(), v.float()

    m, v = series(4 * batch)
    if layer == "delta":
        model, places = DeltaLayer(Nm, max(1, channels // 16), 16, 16, Nd), (9, max(1, channels // 16), 16, 16)
    else:
        model, places = RecurrentLayer(Nm, channels, Nd), (9, channels)
    optimizer = torch.optim.Adam(model.parameters(), lr=5e-3)
    schedule = torch.optim.lr_scheduler.CosineAnnealingLR(optimizer, iterations)
    for i in range(iterations):
        pick = slice(i % 4 * batch, (i % 4 + 1) * batch)
        loss = torch.nn.functional.mse_loss(model(m[pick])[0], v[pick]) / v.square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        schedule.step()
        if report and (i % 100 == 0 or i == iterations - 1):
            report(f"iteration {i}: relative error {loss.item() ** 0.5:.4f}")

    # fresh series, step by step in a cache with more places than streams
    m, v = series(4)
    with torch.no_grad():
        whole, last = model(m)
    state = torch.zeros(places, device="cuda")
    slots = torch.tensor([7, 0, 3, 5], dtype=torch.int32, device="cuda")
    streamed = torch.stack([model.step(m[:, t], state, slots) for t in range(Nt)], 1)
    plan.close()

    def off(x, ref):
        return float((x - ref).norm() / ref.norm())

    result = {"fit": off(whole, v), "stream_against_series": off(streamed, whole),
              "state_against_series": off(state[slots.long()], last)}
    if report:
        report(f"fresh series against F: {result['fit']:.4f}; streamed against the whole series: "
               f"{result['stream_against_series']:.2e}")
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description="fit a recurrent layer to a block Toeplitz operator and stream with it")
    ap.add_argument("--iterations", type=int, default=400)
    ap.add_argument("--steps", type=int, default=200, help="time steps of a series (Nt)")
    ap.add_argument("--layer", choices=["recurrent", "delta"], default="recurrent")
    a = ap.parse_args()
    run(iterations=a.iterations, Nt=a.steps, layer=a.layer)
