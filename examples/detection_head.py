"""A small trainable detection head, from feature maps to suppressed boxes.

  features [batch, rows * columns, channels] (channels last)
    -> 1 x 1 projection -> group norm + SiLU + dropout            (tower)
    -> predictions of (cx, cy, w, h, objectness, classes) per cell
    -> the strongest cells attend to one another with a learned bias by their
       relative position, and are scored again                    (relation)
    -> decode_boxes7 -> boxes7_nms                                (inference)

Trains for a few steps on synthetic maps (a bright spot per object) and runs
the suppression on what it predicts.  `python examples/detection_head.py`.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import greedy_iou_nms_gb300 as g  # noqa: E402
from greedy_iou_nms_gb300 import autograd as ops  # noqa: E402


class Head(torch.nn.Module):
    def __init__(self, channels=64, hidden=128, classes=4, heads=4, reach=7, p=0.1):
        super().__init__()
        self.groups, self.classes, self.heads, self.p = hidden // 8, classes, heads, p

        def weights(*shape):
            return torch.nn.Parameter(torch.randn(*shape) / shape[0] ** 0.5)

        self.tower, self.predict = weights(channels, hidden), weights(hidden, 5 + classes)
        self.norm_weight = torch.nn.Parameter(torch.ones(hidden))
        self.norm_bias = torch.nn.Parameter(torch.zeros(hidden))
        self.qkv, self.join, self.score = weights(hidden, 3 * hidden), weights(hidden, hidden), weights(hidden, 1)
        lut = g.relation_lut_cells(reach, reach)
        self.register_buffer("lut", lut)
        self.table = torch.nn.Parameter(torch.zeros((2 * reach + 1) ** 2, heads))  # a bias by offset and head

    def forward(self, features, side, candidates, seed):
        """Cell logits [B, cells, 5 + classes], the strongest cells' indices and
        their scores after the relation [B, candidates].  seed: of the
        dropout masks of this step (training); None turns them off."""
        p, seed = (0.0, 0) if seed is None else (self.p, seed)
        x = ops.group_norm_act(features @ self.tower, self.groups, self.norm_weight, self.norm_bias, act="silu", p=p,
                               seed=seed, offset=0)
        logits = x @ self.predict
        cells = logits[..., 4].topk(candidates).indices
        picked = torch.gather(x, 1, cells[..., None].expand(-1, -1, x.shape[-1]))
        where = torch.stack([cells // side, cells % side], -1).to(torch.int32)
        buckets = g.relation_buckets(where, where, self.lut)
        B, n, C = picked.shape
        q, k, v = (picked @ self.qkv).view(B, n, 3, self.heads, C // self.heads).permute(2, 0, 3, 1, 4)
        weights = ops.relation_softmax(q @ k.transpose(-1, -2), self.table, buckets, scale=(C // self.heads) ** -0.5)
        weights = ops.dropout(weights, p, seed, 1)
        mixed = (weights @ v).transpose(1, 2).reshape(B, n, C) @ self.join
        picked = ops.dropout(mixed, p, seed, 2, residual=picked)
        return logits, cells, (picked @ self.score)[..., 0]


def batch(generator, size, side, channels, classes):
    """Feature maps with a spot of one class' channels at each of some cells,
    and the cells' targets."""
    features = torch.randn(size, side, side, channels, generator=generator) * 0.3
    target = torch.zeros(size, side, side, dtype=torch.long)
    for b in range(size):
        for _ in range(6):
            r, c = (int(v) for v in torch.randint(1, side - 1, (2,), generator=generator))
            kind = int(torch.randint(0, classes, (1,), generator=generator))
            features[b, r - 1:r + 2, c - 1:c + 2, kind::classes] += 0.7
            features[b, r, c, kind::classes] += 1.0
            target[b, r, c] = kind + 1
    return features.view(size, side * side, channels), target.view(size, -1)


def main(steps=40, size=8, side=20, channels=64, classes=4, candidates=50, device="cuda"):
    g.build()
    torch.manual_seed(0)
    generator = torch.Generator().manual_seed(1)
    model = Head(channels, classes=classes).to(device)
    optimiser = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for step in range(steps):
        features, target = (v.to(device) for v in batch(generator, size, side, channels, classes))
        logits, cells, scores = model(features, side, candidates, seed=step + 1)
        object_here = (target > 0).float()
        bce = torch.nn.functional.binary_cross_entropy_with_logits
        loss = bce(logits[..., 4], object_here, pos_weight=torch.tensor(20.0, device=device))
        loss = loss + bce(scores, torch.gather(object_here, 1, cells))
        kinds = torch.nn.functional.cross_entropy(logits[..., 5:].flatten(0, 1), (target - 1).clamp(min=0).flatten(),
                                                  reduction="none")
        loss = loss + (kinds * object_here.flatten()).sum() / object_here.sum()
        optimiser.zero_grad()
        loss.backward()
        optimiser.step()
        losses.append(loss.detach())
    with torch.no_grad():
        features, target = (v.to(device) for v in batch(generator, size, side, channels, classes))
        logits, cells, scores = model(features, side, candidates, seed=None)
        # Boxes of a fixed size about their cells; objectness of the candidates after the relation, 0 elsewhere.
        preds = torch.zeros(size, side * side, 5 + classes, device=device)
        at = torch.arange(side * side, device=device)
        preds[..., 0], preds[..., 1] = 32.0 * (at % side) + 16, 32.0 * (at // side) + 16
        preds[..., 2:4] = 80.0
        preds[..., 4].scatter_(1, cells, torch.sigmoid(scores))
        preds[..., 5:] = logits[..., 5:].softmax(-1)
        buffers = g.boxes7_nms(g.decode_boxes7(preds, conf_thr=0.25, max_objects=candidates), classes, 0.45)
    found = buffers[:, 0].long()
    kept = buffers[:, 1:].view(size, candidates, 7)[..., 6].sum(1).long()
    return torch.stack(losses).cpu(), found.cpu(), kept.cpu(), model


if __name__ == "__main__":
    losses, found, kept, _ = main()
    print("loss: first", round(float(losses[0]), 3), "last", round(float(losses[-1]), 3))
    print("candidates per image:", found.tolist(), "kept:", kept.tolist())
