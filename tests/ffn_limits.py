"""Error limits of the feed-forward products that are tight enough to see a missing part of the work.

fp32 products are six products of bf16 parts, summed on the tensor cores in steps of four k-blocks.  Of a
step's additions the 16 of the leading parts decide: each is cut off by at most 2^-23 of the sum so far,
which grows like the square root, 2/3 of the step's result on average: 16 * 2/3 * 2^-23 = 1.3e-6 of the
result if every addition lost the most it can, half of that on average.  The steps are added in fp32
(2^-24 sqrt(steps)), and the three part products that are left out by design are below 2^-24 together.
Leaving out any of the six costs 2.4e-6 and more.  So for one product: F32 = 1.2e-6 of the result's
norm; where two products' errors meet (a gate, or a gradient whose operand is a product) sqrt(2) of it.
Single elements of a large result are 5 to 6 standard deviations off: 8 times the limit relative to
the element and the results' rms together, far below what a value that was not written is off.

bf16 rounds by at most 2^-8 of the value (half its spacing of 2^-7).  Forward results are rounded once: every
element within 2^-8 of itself plus 2^-8 of the rms, which covers the fp32 sums under it many times.
Gradients have an operand that was rounded too: a sum of terms each off by at most 2^-8 of itself, with a
standard deviation of at most 2^-8 / sqrt(3) of the root of the terms' squares T.  Seven of those are
2^-6 T, which is also the worst that up to 16 terms can give; on top comes the result's rounding: every
element within 2^-8 of itself plus 2^-6 T.
"""

F32 = 1.2e-6
F32_TWO = 1.7e-6
BF16 = 2.0 ** -8
BF16_TERMS = 2.0 ** -6
