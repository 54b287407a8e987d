"""Clipping in the row-sharded step with two processes (gloo, CPU): the ranks'
sums of squares are gathered between the norm and the update, every rank gets
the same norm and factor, and nothing is clipped unless asked."""
import math
import os
import tempfile

import pytest
import torch
import torch.multiprocessing as mp

from bit_quantization_aware_b200.sharded import LocalPeers, ShardedQuantStep
from tests.test_sharded_order_cpu import MATS, HostLib, ShmPeers, _free_port


class ClipLib(HostLib):
    """The host stand-in with the norm: the plain reduced gradient's squares."""

    @staticmethod
    def pq_grad_norm_workspace_bytes(n, mats=0):
        return 64

    @staticmethod
    def _sums(sources, mult, s):
        n, o = s["rows"] * s["cols"], s["g_offset"]
        acc = torch.zeros(n)
        for src in sources:
            acc += src[o:o + n].float()
        return acc * mult

    @classmethod
    def pq_reduce_grad_norm(cls, q, sources, mult, shards, max_norm, norm, coef, ws, sumsq_out=None, stream=None):
        assert norm is None and coef is None and ws.numel() == 64
        sumsq_out[0] = sum(float(cls._sums(sources, mult, s).double().square().sum()) for s in shards)

    @staticmethod
    def pq_clip_coef(sumsq, max_norm, norm, coef, stream=None):
        norm[0] = math.sqrt(float(sumsq.sum()))
        coef[0] = min(1.0, max_norm / (float(norm) + 1e-6))

    @classmethod
    def pq_reduce_bwd_adamw(cls, q, sources, mult, shards, hp_w, hp_a, stream=None, coef=None):
        for s in shards:
            s["w"].view(-1)[:] = cls._sums(sources, mult, s) * (1.0 if coef is None else float(coef))


def _gradient(rows, rank):
    return (rank + 1) * (torch.arange(rows) % 7 + 1).float()


def _norm(world):
    mean = sum(k + 1 for k in range(world)) / world
    return math.sqrt(sum(float((mean * (torch.arange(m.rows) % 7 + 1)).double().square().sum()) * m.cols for m in MATS))


def _worker(rank, world, port, root, out):
    import torch.distributed as dist
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        st = ShardedQuantStep(MATS, 3, rank, world, ShmPeers(root, rank), device="cpu", lib=ClipLib)
        dist.barrier()
        for i, m in enumerate(MATS):
            st.load_full(i, torch.zeros(m.rows, m.cols), torch.ones(m.rows))
            st.g(i).copy_(_gradient(m.rows, rank)[:, None].expand(m.rows, m.cols))

        def gather(sumsq):
            parts = torch.zeros(world, dtype=torch.float64)
            dist.all_gather_into_tensor(parts, sumsq)
            return parts

        norm = st.backward(dist.barrier, None, None, max_norm=10.0, gather=gather)
        mean = sum(k + 1 for k in range(world)) / world
        coef = torch.tensor(10.0 / (_norm(world) + 1e-6), dtype=torch.float64).float()
        ok = True
        for i, m in enumerate(MATS):
            b, e = st.my_rows(i)
            want = mean * (torch.arange(b, e) % 7 + 1).float() * float(coef)
            # the factor is one fp32 rounding off at most
            ok &= torch.allclose(st.w_shard(i), want[:, None].expand(e - b, m.cols), rtol=2.0 ** -22, atol=0)
        out.put((rank, float(norm), ok))
        dist.barrier()
    finally:
        dist.destroy_process_group()


def test_every_rank_clips_by_the_global_norm():
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    with tempfile.TemporaryDirectory() as root:
        procs = [ctx.Process(target=_worker, args=(r, 2, port, root, q)) for r in range(2)]
        for p in procs:
            p.start()
        res = sorted(q.get(timeout=120) for _ in procs)
        for p in procs:
            p.join(timeout=60)
            assert p.exitcode == 0
    assert [(r, ok) for r, _, ok in res] == [(0, True), (1, True)]
    assert res[0][1] == res[1][1] == pytest.approx(_norm(2), rel=2.0 ** -23)


def test_one_rank_needs_no_gather_and_more_do():
    st = ShardedQuantStep(MATS, 3, 0, 1, LocalPeers(1), device="cpu", lib=ClipLib)
    for i, m in enumerate(MATS):
        st.g(i).copy_(_gradient(m.rows, 0)[:, None].expand(m.rows, m.cols))
    assert float(st.backward(lambda: None, None, None, max_norm=1.0)) == pytest.approx(_norm(1), rel=2.0 ** -23)
    assert st.backward(lambda: None, None, None) is None
    two = ShardedQuantStep(MATS, 3, 0, 2, LocalPeers(2), device="cpu", lib=ClipLib)
    with pytest.raises(ValueError, match="gather"):
        two.clip_coef(1.0)
