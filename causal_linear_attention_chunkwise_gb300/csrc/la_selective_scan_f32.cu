// la_selective_scan_f32.cu -- the selective scan's kernels for fp32 activations.
#define LA_SELECTIVE_SCAN_F32
#include "la_selective_scan.cu"
