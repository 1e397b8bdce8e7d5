"""The barrier protocol of the kernel of many query rows over the 4-bit history, as
test_history_protocol runs it, and what its roles read of a tile's record: the MMA
warp the kind of its second product, between V's arrival and that product.  (The
softmax warps read theirs before they hand over P, which that product waits for.)"""
import pytest

from test_history_protocol import Model


class RecordModel(Model):
    def __init__(self, segments, seed):
        super().__init__(segments, seed)
        self.used = 0

    def hardware(self):
        # read before the product is issued, so also before it runs
        if self.mma and self.mma[0][0] == "pv":
            assert self.record[self.mma[0][2] % 4] == self.mma[0][2]
            self.used += 1
        super().hardware()


@pytest.mark.parametrize("segs", [
    [(1, True, False)], [(3, True, False), (1, True, True)],
    [(5, False, True), (1, True, False), (2, False, False), (7, True, True)], [(6, False, False), (6, True, True)],
])
def test_records_stay_until_the_second_product(segs):
    for seed in range(12):
        m = RecordModel(segs, seed)
        m.run()
        assert m.used == sum(T * (2 if has1 else 1) for T, has1, _ in segs)
