// qc_attend_rows.cuh for heads of 128.
#define QC_ROWS_D 128
#include "qc_attend_rows.cuh"
