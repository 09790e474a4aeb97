"""How the tensor-core kernels end (no device needed; read from their sources).  A wait that runs out may end one warp
role long before the others, and a CTA must not give up its tensor and shared memory while MMAs or copies of its
own still use them: the issuing warp waits for its last MMAs whether or not it gave up itself, and a CTA pair in which a
wait ran out pauses for the copies that nobody counts."""
import os
import re

import pytest

import structured_sparse_transformer_b200 as sp

CSRC = os.path.join(os.path.dirname(os.path.abspath(sp.__file__)), "csrc")
KERNELS = [("gemm_sp.cuh", "sp24_gemm_pair_kernel", True), ("gemm_i8.cuh", "gemm_i8_kernel", True), ("gemm_i8.cuh", "gemm_i8_few_kernel", False),
           ("ortho_gemm.cuh", "orth_products_kernel", True), ("ortho_gemm.cuh", "orth_small_kernel", True),
           ("ortho_gemm.cuh", "orth_last_kernel", True)]


def _body(file, kernel):
    text = open(os.path.join(CSRC, file)).read()
    at = re.search(rf"\b{kernel}\(const __grid_constant__", text).end()
    end = text.index("\n}\n", at)
    return text[at:end]


@pytest.mark.parametrize("file,kernel,pair", KERNELS)
def test_the_issuing_warp_waits_for_its_last_mmas(file, kernel, pair):
    body = _body(file, kernel)
    issuer = body[body.index("else if (warp == 1"):]
    issuer = issuer[:issuer.index("\n  } else if (warp >= 2")]
    last = re.findall(r"^( *)mbar_wait_bounded\((?:drain|over), 0, kDrainBudget", issuer, re.M)
    assert last == ["    "], "one wait, at the level of the role's own statements"
    assert issuer.index("kDrainBudget") > max(m.start() for m in re.finditer(r"tc_commit", issuer))


@pytest.mark.parametrize("file,kernel", [(f, k) for f, k, pair in KERNELS if pair])
def test_a_pair_that_gave_up_pauses_before_it_ends(file, kernel):
    tail = _body(file, kernel)[-500:]
    assert re.search(r"__syncthreads\(\);\s*pair_abort_pause\(s_abort\);\s*cluster_sync\(\);", tail)


def test_no_tensor_memory_is_held_across_a_clusters_wait():
    """A cluster whose CTAs need tensor memory one by one: one that holds it and waits for the others, while another kernel's
    CTAs hold theirs and wait for it, would wait for good.  It is given back before the first wait of the cluster.  (The
    CTA pairs of the other kernels hold it together: their shared memory leaves no room beside them on an SM.)"""
    body = _body("gemm_i8.cuh", "gemm_i8_few_kernel")
    issuer = body[body.index("else if (warp == 1"):body.index("else if (warp >= 2")]
    assert "cluster_sync()" not in issuer and issuer.index("tmem_dealloc(") < issuer.index("cluster_wait()")
    assert body.count("tmem_dealloc(") == 2 and "if (warp == 1 && split == 1)" in body
