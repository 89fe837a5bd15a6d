"""Pin of the oracle's routing: an expert that its bias closes keeps its share of the softmax, one that its score
closes has none."""
import numpy as np

from oracle import router


def test_closed_by_the_score_or_by_the_bias():
    x = np.log(np.array([[2.0, 3.0, 5.0]]))
    ch, w = router.choose(x[0], 2, bias=[0.0, 0.0, -np.inf], renorm=False)
    assert ch == [1, 0] and np.allclose(w, [0.3, 0.2], rtol=1e-15)
    ch, w = router.choose(x[0], 3, bias=[0.0, 0.0, -np.inf])
    assert ch == [1, 0, -1] and np.allclose(w, [0.6, 0.4, 0.0], rtol=1e-15)
    x[0, 2] = -np.inf
    ch, w = router.choose(x[0], 2, bias=[0.0, 0.0, 0.0], renorm=False)
    assert ch == [1, 0] and np.allclose(w, [0.6, 0.4], rtol=1e-15)


def test_the_scale_is_taken_as_it_is():
    assert router.choose([0.0, 0.0], 2, scale=0.1)[1] == [0.05, 0.05]
