"""CPU checks of the long contexts' inputs: a page or key tile that is lost or counted twice anywhere fails the
comparison that the GPU tests make."""
import pytest
import torch

import dense_mla_marked as marked


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("n,dims", [(131072, 512), (215001, 512), (40000, 128), (60001, 128)])
def test_a_lost_or_repeated_page_fails_the_check(n, dims, flat):
    pages = (n + 63) // 64
    level, marker, gain = marked.levels(pages, flat), marked.marker_of(pages, dims), marked.gain_of(10.0, 192 ** -0.5)
    w, lse = marked.weights([n], level, gain)
    want = marked.outputs(w, marker, dims)
    rounded = want.to(torch.bfloat16)
    marked.check(rounded, lse.float(), want, lse)
    for at in list(range(0, pages - 1, 97)) + [pages - 2]:
        for width in (1, 2):
            for times in (0.0, 2.0):
                bad = w.clone()
                bad[:, at:at + width] *= times
                total = bad.sum(1, keepdim=True)
                got = marked.outputs(bad / total, marker, dims).to(torch.bfloat16)
                with pytest.raises(AssertionError, match="out"):
                    marked.check(got, lse.float(), want, lse)
                share = float((total - 1).abs())
                if share > 3 * marked.LSE:
                    with pytest.raises(AssertionError, match="lse"):
                        marked.check(rounded, (lse + torch.log(total[:, 0])).float(), want, lse)
