"""Attention right behind the kernels that write its block tables, on one stream and
without a wait of the host between: such a kernel lets the next one start early, which
must not see the tables as they were before (kept by an SM from the call in front)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
D, BS = 128, 16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Step:
    """n sequences of `rows` query rows, in two sets of blocks with different keys."""

    def __init__(self, n, width, rows, fp8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        hq, hkv = 32, 4
        shared = width // 2
        used = shared + n * (width - shared)
        self.nb = nb = 2 * used
        order = rng.permutation(nb)
        at = np.concatenate([np.tile(np.arange(shared), (n, 1)),
                             shared + np.arange(n * (width - shared)).reshape(n, -1)], axis=1)
        lo, hi = np.sort(order[:used]), np.sort(order[used:])
        self.here, self.there = i32(lo), i32(hi)
        self.tables = i32(lo[at])
        self.first = self.tables.clone()
        lens = rng.integers((width - 1) * BS + 1, width * BS + 1, n)
        self.lens = i32(lens)
        self.k, self.v = (torch.randn(nb, hkv, BS, D, generator=g, device="cuda") for _ in range(2))
        self.ks = self.vs = None
        if fp8:
            self.ks = self.vs = torch.full((hkv,), 1 / 64, device="cuda")
            self.k, self.v = ((x * 64).to(torch.float8_e4m3fn).view(torch.uint8) for x in (self.k, self.v))
        else:
            self.k, self.v = self.k.to(torch.bfloat16), self.v.to(torch.bfloat16)
        self.latents = torch.randn(nb, BS, 576, generator=g, device="cuda").to(torch.bfloat16)
        self.n, self.rows, self.hq = n, rows, hq
        self.cu = i32(np.arange(n + 1) * rows)
        self.q = torch.randn(n * rows, hq, D, generator=g, device="cuda").to(torch.bfloat16)
        self.chunk_q = torch.randn(n * 40, hq, D, generator=g, device="cuda").to(torch.bfloat16)
        self.latent_q = torch.randn(n * rows, hq, 576, generator=g, device="cuda").to(torch.bfloat16)
        self.prefix, self.groups = i32([shared * BS]), i32([0, n])
        self.own = (width - shared) * BS
        self.child = [torch.empty_like(self.tables)] + [i32(np.zeros(n)) for _ in range(3)] + [i32([0])]
        self.parents, self.free = i32(rng.integers(0, n, n)), i32(rng.integers(0, nb, n))

    def chunk(self, tables, lens):
        out = torch.empty(self.chunk_q.shape, device="cuda")
        return pkv.paged_attention_chunked_prefill(out, self.chunk_q, self.cu * (40 // self.rows), lens, 40, self.k, self.v, tables,
                                                   k_scale=self.ks, v_scale=self.vs)

    def drafts(self, tables, lens):
        if self.rows == 1:
            out = torch.empty(self.q.shape, device="cuda")
            return pkv.paged_attention_decode(out, self.q, self.k, self.v, tables, lens, D ** -0.5, self.ks, self.vs)
        out = torch.empty(self.q.shape, device="cuda")
        return pkv.paged_attention_chunked_prefill(out, self.q, self.cu, lens, self.rows, self.k, self.v, tables,
                                                   k_scale=self.ks, v_scale=self.vs)

    def shared(self, tables, lens):
        # (after a fork the children's tails have not come from one parent, but the prefix has)
        return pkv.paged_attention_shared_prefix(
            torch.empty_like(self.q), self.q, self.k, self.v, tables, lens, self.groups, self.prefix,
            cu_q_lens=self.cu, max_q_len=self.rows, max_prefix_len=int(self.prefix_len), max_tail_len=self.own,
            k_scale=self.ks, v_scale=self.vs)

    def latent(self, tables, lens):
        out = torch.empty(self.n * self.rows, self.hq, 512, device="cuda", dtype=torch.bfloat16)
        return pkv.paged_latent_attention(out, self.latent_q, self.latents, tables, lens, cu_q_lens=self.cu)

    @property
    def prefix_len(self):
        return self.first.shape[1] // 2 * BS

    def pass_(self, attend, wait):
        """The tables' blocks move there and back, twice, and the sequences fork, each followed by `attend`."""
        sync = torch.cuda.synchronize if wait else (lambda: None)
        outs = []
        for _ in range(2):
            for src, dst in ((self.here, self.there), (self.there, self.here)):
                outs.append(attend(self.tables, self.lens))
                sync()
                pkv.kv_remap_tables(self.tables, self.lens, src, dst)
                sync()
                outs.append(attend(self.tables, self.lens))
                sync()
            pkv.kv_fork_tables(self.tables, self.lens, self.parents, self.free, *self.child)
            sync()
            outs.append(attend(self.child[0], self.child[1]))
            sync()
        assert torch.equal(self.tables, self.first)
        return outs


@pytest.mark.parametrize("n,width,rows", [(6, 8, 1), (64, 64, 1), (24, 40, 4)])
@pytest.mark.parametrize("call,fp8", [("chunk", False), ("chunk", True), ("drafts", False), ("drafts", True),
                                      ("shared", False), ("shared", True), ("latent", False)])
def test_attention_right_behind_the_tables(call, n, width, rows, fp8):
    s = Step(n, width, rows, fp8)
    attend = getattr(s, call)
    apart = [x.clone() for x in s.pass_(attend, wait=True)]
    assert not torch.equal(apart[0], apart[1])       # (the two sets of blocks do differ)
    for _ in range(5):
        for a, b in zip(apart, s.pass_(attend, wait=False)):
            assert torch.equal(a, b)
    assert pkv.kv_last_device_status() == 0
