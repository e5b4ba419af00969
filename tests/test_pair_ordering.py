"""Memory ordering between the two CTAs of a pair, read from the kernels' sources.

A pair's leader issues the tcgen05.cp that reads both CTAs' code tiles.  Where
warps wrote those with plain stores, the peer's arrival has to release at
cluster scope and the leader's wait to acquire at cluster scope: the default
scope is the CTA, which orders nothing between the two.  A run cannot show the
ordering (it may come right by chance), so the sources are read."""
import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "structured_sparse_pretraining_b200", "csrc")

# sources in which warps of both CTAs write codes that the leader's tcgen05.cp reads
Q8_PAIRS = ["gemm_q8_pair.cuh", "gemm_q8_wide.cuh"]


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", Q8_PAIRS)
def test_codes_of_the_peer_are_released_and_acquired_at_cluster_scope(name):
    text = source(name)
    # a remote arrival on `full` (bytes of TMA apart) is the relay's alone
    assert not re.search(r"mbar_arrive_cluster\w*\(cluster_addr\(&full\[", text)
    assert "q8_relay_codes<NS>(codes, full" in text and "mbar_wait_codes(&full[" in text
    relay = re.search(r"bool q8_relay_codes\(.*?\n}", source("gemm_q8.cuh"), re.S).group(0)
    assert relay.index("mbar_wait_warp(&codes[s]") < relay.index("mbar_arrive_cluster_rel(cluster_addr(&full[s], 0))")


@pytest.mark.parametrize("name", ["gemm_pair.cuh", "gemm_wide.cuh"])
def test_lane_images_of_the_peer_are_released_and_acquired_at_cluster_scope(name):
    """The bf16 products' code tiles, rearranged in place by warps of both CTAs."""
    text = source(name)
    assert not re.search(r"mbar_arrive_cluster\w*\(cluster_addr\(&mfull\[e", text)
    assert re.search(r"relay_codes<\w+>\(mpeer, mfull", text)
    waits = re.findall(r"(mbar_wait\w*)\(&mfull\[", text)
    assert waits and set(waits) == {"mbar_wait_cluster"}, waits
    relay = re.search(r"bool relay_codes\(.*?\n}", source("gemm_pair.cuh"), re.S).group(0)
    assert relay.index("mbar_wait(&mpeer[b]") < relay.index("mbar_arrive_cluster_rel(cluster_addr(&mfull[b], 0))")


def test_the_helpers_name_the_cluster():
    text = source("ptx.cuh")
    body = lambda name: re.search(name + r"\(.*?\n}", text, re.S).group(0)  # noqa: E731
    assert "mbarrier.arrive.release.cluster.shared::cluster" in body("void mbar_arrive_cluster_rel")
    assert "mbarrier.try_wait.parity.acquire.cluster" in body("bool mbar_wait_cluster")
    assert "mbar_wait_cluster(" in body("bool mbar_wait_codes")


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,M,form", [(1024, 1984, 4160, 256), (4000, 1472, 2752, 256), (3300, 832, 1984, 512), (2222, 5824, 2880, 512)])
def test_codes_without_tma_change_from_call_to_call(T, K, M, form):
    """K an odd multiple of 64 in the pair forms: stages that held other codes a moment before."""
    import q8_plain as P
    from structured_sparse_pretraining_b200 import ops
    assert ops.q8_plan(M, T, K, 0)[0] == form
    Xq, Wq = P.random_int8(T, K, 1), P.random_int8(M, K // 2, 2)
    xs, ws = torch.full((T,), 2.0 ** -6, device="cuda"), torch.full((M,), 2.0 ** -9, device="cuda")
    metas = [P.random_codes(M, K, s) for s in (3, 4, 5)]
    wants = [P.product(Xq, xs, Wq, ws, m) for m in metas]
    outs = [ops.fwd_q8(Xq, xs, Wq, ws, metas[i % 3], None, None, M) for i in range(24)]
    ops.status_sync()
    for i, y in enumerate(outs):
        want, tol = wants[i % 3]
        assert ((y.double() - want).abs() <= tol).all(), i
