"""Learns labels of a scene's Gaussians from a part of them, and names the rest.

Gaussians that lie together share a code (a cell of a grid over the scene), as
after vector quantisation of their features. A few of them carry a label. The
label head (codebook lookup, layer normalisation, vocabulary loss) is trained
on those and then asked for the others.

    python examples/label_scene.py [--gaussians N] [--steps N] [--dtype float32|bfloat16]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from differentiable_gaussian_splat_amd import labels, scenes  # noqa: E402


def cells(means, per_axis):
    """Code of each Gaussian: its cell in a grid with as many Gaussians in each slab of an axis."""
    code = np.zeros(means.shape[0], dtype=np.int64)
    for axis in range(3):
        rank = np.argsort(np.argsort(means[:, axis], kind="stable"), kind="stable")
        code = code * per_axis + rank * per_axis // means.shape[0]
    return code


def train(n=50_000, steps=60, dim=64, vocabulary=40, per_axis=12, labelled=0.1, dtype=torch.float32, seed=0):
    """Trains a head; returns (first loss, last loss, share of the unlabelled Gaussians named rightly)."""
    dev = torch.device("cuda")
    torch.manual_seed(seed)
    codes = torch.from_numpy(cells(scenes.make_scene(3, seed, n=n).means, per_axis)).to(dev)
    truth = torch.randint(0, vocabulary, (per_axis ** 3,), device=dev)[codes]  # a cell is of one thing
    known = torch.rand(n, device=dev) < labelled
    given = torch.where(known, truth, -1)
    head = labels.LabelHead(per_axis ** 3, dim, vocabulary, device=dev, dtype=dtype)
    opt = torch.optim.Adam(head.parameters(), lr=2e-2)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = head(codes, given)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    with torch.no_grad():
        every = torch.arange(per_axis ** 3, device=dev)
        name = (head.features(every).float() @ head.vocabulary.float().t()).argmax(1)
        right = (name[codes] == truth)[~known].float().mean()
    return float(losses[0]), float(losses[-1]), float(right)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--gaussians", type=int, default=50_000)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=["float32", "bfloat16"], default="float32")
    a = ap.parse_args()
    first, last, right = train(a.gaussians, a.steps, dtype=getattr(torch, a.dtype))
    print(f"loss {first:.4f} -> {last:.4f} over {a.steps} steps; {100 * right:.1f} % of the unlabelled Gaussians named")


if __name__ == "__main__":
    main()
