"""The ends of the serving entry points' ranges, on the host: calls that fail validation,
with addresses that nothing reads."""
from test_abi_serving import ERR_ARG, ERR_SHAPE, D, P, refused  # noqa: F401


def test_token_logprobs_rows(D):  # noqa: F811
    """2^24 rows of 256 threads are one work-item more than a launch can have."""
    L = D.lib()

    def call(N, logits):
        return L.dspark_token_logprobs(1, N, 2, 2, logits, P, 1, P, P, P, P, P, 1 << 30, None)

    refused(D, ERR_SHAPE, call(2 ** 24, P))
    refused(D, ERR_ARG, call(2 ** 24 - 1, None))
    assert L.dspark_logprobs_workspace_bytes(2 ** 24, 1 << 20, 1) == 0
