"""The failure report of attention over prompts and of drafted trees, without a GPU fault: a bounded wait of each family of
kernels runs out, gdn_attn_device_status names it once, and calls go on as before."""
import pytest
import torch

pytestmark = pytest.mark.gpu
NAMES = ["prompt forward", "prompt backward", "tree bf16", "tree 8 bits"]


@pytest.fixture(scope="module", autouse=True)
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build, gdn
    build.build()
    assert gdn.gdn_attn_device_status() == gdn.GDN_OK
    return gdn


def works(gdn):
    x = torch.ones(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    o = gdn.prompt_attention(x, x, x)
    assert gdn.gdn_attn_device_status() == gdn.GDN_OK and torch.equal(o, x)


@pytest.mark.parametrize("kernels", range(4))
def test_a_wait_that_runs_out_is_reported_once(gdn, kernels):
    gdn.gdn_debug_attn_wait_timeout(kernels, 2000)  # gives up after 2 ms
    assert gdn.gdn_attn_device_status() == gdn.GDN_ERR_TIMEOUT
    word = NAMES[kernels].split()
    text = gdn.lib().gdn_last_error().decode()
    prompt, tree = text[text.index("(prompt"):].rstrip(")").split(", tree")
    assert (prompt[1:] + "|tree" + tree).split("|")[0 if word[0] == "prompt" else 1] == NAMES[kernels]
    assert (prompt[1:], "tree" + tree)[1 if word[0] == "prompt" else 0] in ("prompt", "tree")  # no other family
    works(gdn)


def test_all_of_them_on_another_stream(gdn):
    side = torch.cuda.Stream()
    for kernels in range(4):
        gdn.gdn_debug_attn_wait_timeout(kernels, 2000, stream=side)
    assert gdn.gdn_attn_device_status(side) == gdn.GDN_ERR_TIMEOUT
    assert "prompt forward backward, tree bf16 8 bits" in gdn.lib().gdn_last_error().decode()
    works(gdn)
