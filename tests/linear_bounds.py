"""Bounds on the errors of the linear attention calls, for inputs of
independent normal numbers and at least a hundred tokens, as relative 2-norms
of a whole output.  They count roundings by their root mean square, where the
bounds of test_gpu_linear.py add the largest possible ones.

bf16 outputs.  A rounding to bf16 is off by at most 2^-8 of the value, evenly
spread: 2^-8 / sqrt(3) of it in the mean square (ROUND) where all values are
just above a power of two, and less elsewhere.  The CUDA cores round once, the
output itself.  The tensor-core path rounds one operand of each product too (the
weighted pairs, or the state), so an output is the sum of two parts whose errors
are independent of each other and of the output's own: sqrt(2) ROUND.

fp32 outputs.  A state is a sum of terms w c b^T; w is a product of at most two
exponentials (2 ulp each, 2^-22 relative) and c times w is rounded (2^-24), so the
terms are off by 2^-21 at the very most, and by less than half of that in the mean
square; the sums over 16 x 8 tokens in the tensor cores, or 256 on the CUDA
cores, and the carries add roundings of 2^-23 of a partial sum each, of which
mostly independent ones come to less than sqrt(32) 2^-24: together below 2^-20,
held to 2^-19.  (A state of which w c has lost its third bf16 term is off by
more: test_linear_split.py.)

The gradient of the decays at a token is a sum over up to 512 tokens of
differences (R - C), each off by up to 2^-22 of its terms, while the sum itself
has the size of those pairs only that the decays leave between both sides of the
token: with a memory of m tokens sqrt(512 / m) times 2^-22.  With m = 12, the
memory of the decays used here, 1.6e-6, held to 2^-18."""
BF16_ROUND = 2.0 ** -8 / 3 ** 0.5
STATE = 2.0 ** -19
DECAYS = 2.0 ** -18


def out_bound(fp32, path):
    return STATE if fp32 else (BF16_ROUND if path == "simt" else 2 ** 0.5 * BF16_ROUND) + STATE
