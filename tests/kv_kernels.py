"""Sends attention calls to a named kernel: which one takes a call goes by the sizes that the host sees, so the table
gets columns that no request reaches, and the hint says how many queries a request has."""
import torch

from lossless_float_weight_amd import zn

KINDS = ("short", "short pairs", "few rows", "many rows")


def widened(table, width):
    """The table with columns of -1 behind its own."""
    wide = torch.full((table.shape[0], max(width, table.shape[1])), -1, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    return wide


def sized(kind, q, c, table, starts):
    """(table, starts, max_new) for a call of these shapes that goes to the kernel; an error if none does."""
    kv_heads, page = c.k.shape[1:3]
    tiles, hint = {"short": (1, 1), "short pairs": (1, 1), "few rows": (40, 1),
                   "many rows": (20480 // kv_heads + 1, q.shape[0])}[kind]
    table = widened(table, -(-tiles * 64 // page))
    if kind == "many rows" and starts is None:
        starts = torch.arange(q.shape[0] + 1, dtype=torch.int32, device=q.device)
    return table, starts, hint


def attention_by(kind):
    """mx_attention by that kernel.  A call whose shapes do not reach it is a fault of the test."""
    attention = zn.mx_attention

    def call(q, c, table, lens, starts=None, max_new=0, **kw):
        table, starts, hint = sized(kind, q, c, table, starts)
        got = zn.debug_attention_kernel(q, c, table, starts, hint, kw.get("window", 0))
        assert got == kind, f"these sizes go to the kernel of {got}, not {kind}"
        return attention(q, c, table, lens, starts, max_new=hint, **kw)
    return call
