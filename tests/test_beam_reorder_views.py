"""beam_reorder moves bytes: states whose values are not their bytes (lazily
conjugated or negated views) are refused."""

import pytest
import torch

from rejection_sampling_verifier_amd import binding


@pytest.mark.parametrize("of", [lambda x: x.conj(), lambda x: x.conj().imag])
def test_lazy_views_are_refused(of):
    state, anc = torch.zeros((4, 3), dtype=torch.complex64), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="resolve"):
        binding.beam_reorder(of(state), anc)
    with pytest.raises(ValueError, match="resolve"):
        binding.beam_reorder(of(state).clone().resolve_conj().resolve_neg(), anc, out=of(state))
    with pytest.raises(ValueError, match="GPU"):
        binding.beam_reorder(of(state).resolve_conj().resolve_neg(), anc)
