"""Windows and first tokens of spec_prompt_attention at the ends of 32 bits: "all of them" is a natural thing to ask for."""

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.test_gpu_prompt_attention import check, make  # noqa: E402

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window,sinks", [(250, MOST), (250, MOST - 8), (250, MOST - 15), (250, MOST - 16), (7, MOST), (1, MOST), (256, MOST), (255, MOST - 1),
                                          (MOST, MOST), (MOST, 0), (MOST - 200, 5), (MOST - 1, MOST)])
def test_all_tokens_stay_visible(window, sinks, dtype):
    # a window's first visible position is not a multiple of 16: the first tile begins in front of the prompt
    check(make(31, [420, 3, 0, 700], 1, 1, 64, dtype), window, sinks)
    check(make(32, [260, 131, 300], 8, 2, 64, dtype), window, sinks)


@pytest.mark.parametrize("window,sinks", [(250, MOST), (60, MOST - 3), (MOST, MOST)])
def test_all_tokens_of_wide_heads_stay_visible(window, sinks):
    check(make(33, [420, 90], 2, 2, 256), window, sinks)
    check(make(34, [300], 7, 1, 128), window, sinks)
