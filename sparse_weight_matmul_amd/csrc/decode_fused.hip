// The decode kernels' instances with an epilogue (launch_decode_fused), a unit
// of its own so that they compile beside those without one.
#define SWM_DECODE_FUSED_UNIT
#include "decode.hip"
