// Test shim: the slices and mbarriers of the distillation gradient's pipeline
// (grad_signals.cuh), compiled for the host so that a CPU test can explore the
// pipeline's signals with the same arithmetic the kernel uses.
#include "grad_signals.cuh"

extern "C" int grad_slice_of(int n) { return dspark::slice_of(n); }
extern "C" int grad_full_of(int n) { return dspark::full_of(n); }
extern "C" int grad_full_parity(int n) { return static_cast<int>(dspark::full_parity(n)); }
